// Per-head RMS norm of queries and keys with the position rotation in the same
// pass, the append of keys and values to a paged cache, the gradient, and the
// table of rotations.
//
// Forward, for one head row x of D elements at position pos, in fp32:
//   n = x w / sqrt(mean(x^2) + eps),   y = R(pos) n,
// where R turns the pairs of the first rot_dim elements by the table's angles
// (pair i is (i, i + rot/2) or (2i, 2i + 1)); y is rounded once, at the store.
// Backward, with u = R^T g and r = 1 / sqrt(mean(x^2) + eps):
//   dw = sum u x r,   dx = r (u w - x r^2 mean(u w x)).
//
// Memory bounds all of them (a row is read once and written once, ~5 flops a
// byte at most), so the work is laid out for wide loads: a row belongs to a
// power-of-two number of lanes, each with two 16-byte vectors that hold both
// halves of its pairs, so that the rotation needs no exchange and the norm one
// shuffle sum.  A group of lanes takes several heads of one token and issues
// their loads together; the angles stay in registers across the heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "sbt_internal.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kThreads = 128;
// Forward: heads per group, and blocks per SM the registers are held to.  30011
// fp16 tokens of 32 + 8 + 8 heads of 128 with 4 heads: 113 us at 7 blocks, 115 at 6, 129
// at 4; with 3 heads 120, with 2 heads 122, with one 188.
constexpr int kFwdHeads = 4, kFwdBlocks = 7;
// Rows per SM and group of lanes from which a group takes several heads, if not more than a
// quarter of the places stay empty.  bf16, 32 + 8 + 8 heads: 256 tokens 3.9 us with four
// heads, 3.1 with one; 512 tokens 4.5 and 4.7; 1024 tokens 6.2 and 7.5.  8 + 1 + 1 heads (four
// leave 6 of 16 places empty): 1024 tokens 4.5 and 3.0, 8192 tokens 12.0 and 11.7.
constexpr int kManyRows = 10;
// Gradient: heads per item, stages of the ring.  16384 bf16 tokens of 32 + 8 heads of 128: 80 us
// with (2, 2); 94 with (1, 2), 99 with (4, 2), 114 with (2, 3).
constexpr int kBwdHeads = 2, kStages = 2;
constexpr int kMaxScalarPairs = 8;  // pairs per lane of the element path: 512 elements

enum Kind { kF32 = 0, kBF16 = 1, kF16 = 2 };

template <int KIND> struct Num;
template <> struct Num<kF32> {
    typedef uint32_t T;
    static constexpr int V = 4;
    static __device__ __forceinline__ float get(uint32_t x) { return __uint_as_float(x); }
    static __device__ __forceinline__ uint32_t put(float x) { return __float_as_uint(x); }
};
template <> struct Num<kBF16> {
    typedef uint16_t T;
    static constexpr int V = 8;
    static __device__ __forceinline__ float get(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
    static __device__ __forceinline__ uint16_t put(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
template <> struct Num<kF16> {
    typedef uint16_t T;
    static constexpr int V = 8;
    static __device__ __forceinline__ float get(uint16_t x) { return __half2float(__ushort_as_half(x)); }
    static __device__ __forceinline__ uint16_t put(float x) { return __half_as_ushort(__float2half_rn(x)); }
};

template <int KIND>
__device__ __forceinline__ void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (KIND == kF32) {
            x[i] = __uint_as_float(w[i]);
        } else if (KIND == kBF16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

template <int KIND>
__device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (KIND == kF32) {
            w[i] = __float_as_uint(x[i]);
        } else if (KIND == kBF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Rows {  // [tokens][heads][D], strides in bytes
    const char* p;
    int64_t ld, ldh;
    __device__ __forceinline__ const char* at(int64_t t, int h) const { return p + t * ld + h * ldh; }
};

struct FwdParams {
    Rows x[3];                // q, k, v
    Rows y[2];                // q_out, k_out (p may be NULL)
    const char* w[2];
    int32_t heads[3];
    int64_t tokens;
    int32_t D, rot, interleaved;
    const int32_t* pos;
    const float2* table;      // [n_pos][rot / 2] (cos, sin)
    int64_t n_pos;
    float eps;
    // cache (k_cache NULL: none); byte strides
    char* cache[2];
    int64_t ld_page, ld_slot, ld_head;
    const int32_t* page_table;
    const int32_t* seq;
    int64_t ld_table, n_pages;
    int32_t n_seq, max_pages;
    sbt_fastdiv page_size;
};

// Byte offset of a token's slot in the cache, or -1 where it has none.
__device__ __forceinline__ int64_t cache_slot(const FwdParams& p, int64_t t, int32_t pos) {
    const int64_t s = p.seq ? (int64_t)sbt_ld(p.seq + t) : t;
    if (s < 0 || s >= p.n_seq || pos < 0) return -1;
    const uint32_t j = sbt_div(p.page_size, (uint32_t)pos);
    if (j >= (uint32_t)p.max_pages) return -1;
    const int32_t page = sbt_ld(p.page_table + s * p.ld_table + j);
    if (page < 0 || page >= p.n_pages) return -1;
    return page * p.ld_page + (int64_t)(pos - (int32_t)(j * p.page_size.d)) * p.ld_slot;
}

// The two vectors of lane j of a row: element offsets (-1: none), and for the
// first V / 2 and the last V / 2 of the lane's V pairs where they start in the
// table (-1: not turned).  Neighbouring lanes hold neighbouring vectors: two
// 16-byte halves of one 32-byte sector in different instructions would cost
// twice the L2 traffic (measured on the fp16 interleaved append: 179 us so).
struct Place {
    int a, b, pair[2];
};
template <int V, bool INTER>
__device__ __forceinline__ Place place_of(int j, int lanes, int D, int rot) {
    Place q;
    if (INTER) {  // vectors j and j + lanes, V / 2 pairs in each
        q.a = j * V < D ? j * V : -1;
        q.b = (lanes + j) * V < D ? (lanes + j) * V : -1;
        q.pair[0] = q.a >= 0 && q.a < rot ? q.a / 2 : -1;
        q.pair[1] = q.b >= 0 && q.b < rot ? q.b / 2 : -1;
        return q;
    }
    const int np = rot / (2 * V);
    if (j < np) {  // pairs jV .. jV + V - 1, one element in each vector
        q.a = j * V;
        q.b = rot / 2 + j * V;
        q.pair[0] = j * V;
        q.pair[1] = j * V + V / 2;
    } else {       // what is not turned: its first half over the lanes left, then the second
        const int left = (D - rot) / V, half = (left + 1) / 2, i = j - np;
        q.a = i < half ? rot + i * V : -1;
        q.b = i < half && half + i < left ? rot + (half + i) * V : -1;
        q.pair[0] = q.pair[1] = -1;
    }
    return q;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_l1(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// cos and sin of this lane's V pairs.
template <int V>
__device__ __forceinline__ void angles(const float2* row, const Place& q, float* cs, float* sn) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const int first = q.pair[i / (V / 4)];
        float4 c = make_float4(1.f, 0.f, 1.f, 0.f);
        if (first >= 0) c = sbt_ld(reinterpret_cast<const float4*>(row + first + 2 * (i % (V / 4))));
        cs[2 * i] = c.x, sn[2 * i] = c.y, cs[2 * i + 1] = c.z, sn[2 * i + 1] = c.w;
    }
}

// Turns the lane's 2 V elements (x[0..V) of vector a, x[V..2V) of vector b); sign -1: the transpose.
// Pairs that are not turned are left alone, not turned by an angle of 0: 0 times an infinite partner is NaN.
template <int V, bool INTER>
__device__ __forceinline__ void turn(float* x, const Place& q, const float* cs, const float* sn, float sign) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (q.pair[i / (V / 2)] < 0) continue;
        const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : V + i;
        const float a = x[ia], b = x[ib], s = sign * sn[i];
        x[ia] = a * cs[i] - b * s;
        x[ib] = b * cs[i] + a * s;
    }
}

template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int d = LPR / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// HB heads of one kind of a token per group: grid (head blocks, token blocks).
template <int KIND, bool INTER, int LPR, int HB>
__global__ void __launch_bounds__(kThreads, HB == 1 ? 1 : kFwdBlocks) k_norm_rope(const FwdParams p) {
    sbt_ptx::griddep_wait();
    constexpr int V = Num<KIND>::V, ES = 16 / V, GROUPS = kThreads / LPR;
    const int j = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const Place at = place_of<V, INTER>(j, LPR, p.D, p.rot);
    const int hq = (p.heads[0] + HB - 1) / HB, hk = (p.heads[1] + HB - 1) / HB;
    const int kind = (int)blockIdx.x < hq ? 0 : (int)blockIdx.x < hq + hk ? 1 : 2;
    const int h0 = (blockIdx.x - (kind >= 1 ? hq : 0) - (kind == 2 ? hk : 0)) * HB;
    const int rows = p.heads[kind] - h0;  // min(rows, HB) of them here
    const Rows in = p.x[kind];
    char* const cache = kind >= 1 ? p.cache[kind - 1] : nullptr;
    const char* const wp = kind < 2 ? p.w[kind] : nullptr;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t t0 = (int64_t)blockIdx.y * GROUPS; t0 < p.tokens; t0 += (int64_t)gridDim.y * GROUPS) {
        const int64_t t = t0 + g;
        const bool on = t < p.tokens;
        const int32_t pos = on ? sbt_ld(p.pos + t) : -1;
        const char* x = in.at(on ? t : 0, h0);
        uint4 va[HB], vb[HB];
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            va[i] = on && i < rows && at.a >= 0 ? *reinterpret_cast<const uint4*>(x + i * in.ldh + at.a * ES) : zero;
            vb[i] = on && i < rows && at.b >= 0 ? *reinterpret_cast<const uint4*>(x + i * in.ldh + at.b * ES) : zero;
        }
        const bool real = pos >= 0 && (p.rot == 0 || pos < p.n_pos);
        int64_t slot = -1;
        if (cache && real) slot = cache_slot(p, t, pos);
        char* y = on && kind < 2 && p.y[kind].p ? const_cast<char*>(p.y[kind].at(t, h0)) : nullptr;
        const int64_t ldy = kind < 2 ? p.y[kind].ldh : 0;
        char* kept = slot >= 0 ? cache + slot + h0 * p.ld_head : nullptr;
        float cs[V], sn[V];
        if (kind < 2) {  // the same for the whole block
            if (p.rot && real) {
                angles<V>(p.table + (int64_t)pos * (p.rot / 2), at, cs, sn);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) cs[i] = 1.f, sn[i] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            uint4 a = va[i], b = vb[i];
            if (kind < 2) {
                float f[2 * V];
                unpack<KIND>(a, f);
                unpack<KIND>(b, f + V);
                if (wp) {
                    float ss = 0.f, w[2 * V];
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) ss += f[e] * f[e];
                    const float r = rsqrtf(lanes_sum<LPR>(ss) / (float)p.D + p.eps);
                    unpack<KIND>(at.a >= 0 ? sbt_ld(reinterpret_cast<const uint4*>(wp + at.a * ES)) : zero, w);
                    unpack<KIND>(at.b >= 0 ? sbt_ld(reinterpret_cast<const uint4*>(wp + at.b * ES)) : zero, w + V);
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) f[e] = f[e] * r * w[e];
                }
                turn<V, INTER>(f, at, cs, sn, 1.f);
                a = real ? pack<KIND>(f) : zero;
                b = real ? pack<KIND>(f + V) : zero;
            }
            if (i < rows && y) {
                if (at.a >= 0) *reinterpret_cast<uint4*>(y + i * ldy + at.a * ES) = a;
                if (at.b >= 0) *reinterpret_cast<uint4*>(y + i * ldy + at.b * ES) = b;
            }
            if (i < rows && kept) {
                if (at.a >= 0) *reinterpret_cast<uint4*>(kept + i * p.ld_head + at.a * ES) = a;
                if (at.b >= 0) *reinterpret_cast<uint4*>(kept + i * p.ld_head + at.b * ES) = b;
            }
        }
    }
}

// Element offsets of pair i: the turned ones first, then what is left, two by two (-1: none).
__device__ __forceinline__ void pair_at(int i, int D, int rot, bool inter, int* a, int* b) {
    if (i < rot / 2) {
        *a = inter ? 2 * i : i;
        *b = inter ? 2 * i + 1 : i + rot / 2;
    } else {
        const int d = rot + 2 * (i - rot / 2);
        *a = d < D ? d : -1;
        *b = d + 1 < D ? d + 1 : -1;
    }
}

// Any alignment and any sizes: one warp per row, element accesses.
template <int KIND>
__global__ void __launch_bounds__(kThreads) k_norm_rope_elems(const FwdParams p) {
    typedef typename Num<KIND>::T T;
    sbt_ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int total = p.heads[0] + p.heads[1] + p.heads[2];
    const int64_t rows = p.tokens * total;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); row < rows;
         row += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t t = row / total;
        int h = (int)(row - t * total);
        const int kind = h < p.heads[0] ? 0 : h < p.heads[0] + p.heads[1] ? 1 : 2;
        h -= (kind >= 1 ? p.heads[0] : 0) + (kind == 2 ? p.heads[1] : 0);
        const int32_t pos = sbt_ld(p.pos + t);
        const bool real = pos >= 0 && (p.rot == 0 || pos < p.n_pos);
        const T* x = reinterpret_cast<const T*>(p.x[kind].at(t, h));
        float a[kMaxScalarPairs], b[kMaxScalarPairs], ss = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxScalarPairs; ++i) {
            int ia, ib;
            pair_at(lane + 32 * i, p.D, p.rot, p.interleaved, &ia, &ib);
            a[i] = ia >= 0 ? Num<KIND>::get(x[ia]) : 0.f;
            b[i] = ib >= 0 ? Num<KIND>::get(x[ib]) : 0.f;
            ss += a[i] * a[i] + b[i] * b[i];
        }
        ss = lanes_sum<32>(ss);
        T* y0 = nullptr;
        T* y1 = nullptr;
        if (kind < 2 && p.y[kind].p) y0 = reinterpret_cast<T*>(const_cast<char*>(p.y[kind].at(t, h)));
        if (kind >= 1 && p.cache[kind - 1] && real) {
            const int64_t slot = cache_slot(p, t, pos);
            if (slot >= 0) y1 = reinterpret_cast<T*>(p.cache[kind - 1] + slot + h * p.ld_head);
        }
        const T* w = kind < 2 ? reinterpret_cast<const T*>(p.w[kind]) : nullptr;
        const float r = w ? 1.f / sqrtf(ss / (float)p.D + p.eps) : 1.f;
#pragma unroll
        for (int i = 0; i < kMaxScalarPairs; ++i) {
            const int pr = lane + 32 * i;
            int ia, ib;
            pair_at(pr, p.D, p.rot, p.interleaved, &ia, &ib);
            float u = a[i], v = b[i];
            if (w) {
                if (ia >= 0) u = u * r * Num<KIND>::get(w[ia]);
                if (ib >= 0) v = v * r * Num<KIND>::get(w[ib]);
            }
            if (kind < 2 && pr < p.rot / 2 && real) {
                const float2 cs = sbt_ld(p.table + (int64_t)pos * (p.rot / 2) + pr);
                const float uu = u * cs.x - v * cs.y;
                v = v * cs.x + u * cs.y;
                u = uu;
            }
            const T ta = real ? Num<KIND>::put(u) : T(0), tb = real ? Num<KIND>::put(v) : T(0);
            if (y0 && ia >= 0) y0[ia] = ta;
            if (y0 && ib >= 0) y0[ib] = tb;
            if (y1 && ia >= 0) y1[ia] = ta;
            if (y1 && ib >= 0) y1[ib] = tb;
        }
    }
}

// -------------------------------------------------------------------------------- backward

struct BwdParams {
    Rows g[2], x[2], dx[2];
    const char* w[2];
    int32_t heads[2];
    int64_t tokens;
    int32_t D, rot, interleaved;
    const int32_t* pos;
    const float2* table;
    int64_t n_pos;
    float eps;
    int32_t blocks[2];   // blocks on queries, on keys
    float* partial;      // [blocks[0] + blocks[1]][D]
    float* dw[2];
};

// Items of the vector kernel: HB heads of one token.  A group of
// LPR lanes walks the items with a fixed stride, so that the place of the next
// one follows by additions.
struct Item {
    int64_t t;
    int32_t hb;
};
__device__ __forceinline__ Item item_at(int64_t i, int32_t hblocks) {
    Item x;
    x.t = i / hblocks;
    x.hb = (int32_t)(i - x.t * hblocks);
    return x;
}
__device__ __forceinline__ void advance(Item& x, const Item& step, int32_t hblocks) {
    x.t += step.t;
    x.hb += step.hb;
    if (x.hb >= hblocks) {
        x.hb -= hblocks;
        ++x.t;
    }
}

// One block takes head rows of the queries or of the keys only, so one set of
// sums for dw stays in registers; the blocks' sums go to the workspace and are
// added in block order by k_norm_rope_dw: no atomics, the same bits every run.
template <int KIND, bool INTER, int LPR, int HB, int STAGES>
__global__ void __launch_bounds__(kThreads) k_norm_rope_bwd(const BwdParams p) {
    constexpr int V = Num<KIND>::V, ES = 16 / V, GROUPS = kThreads / LPR, AV = V / 2;
    constexpr int VECS = 4 * HB + AV;
    extern __shared__ __align__(16) uint8_t smem[];  // [STAGES][VECS][kThreads] vectors, positions; then the sums
    uint4* const ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;
    int32_t* const s_pos = reinterpret_cast<int32_t*>(smem + (size_t)STAGES * VECS * kThreads * 16) + threadIdx.x;
    float* const s_dw = reinterpret_cast<float*>(smem);  // [GROUPS][LPR * 2 V], after the last item
    const uint32_t ring_u32 = sbt_ptx::smem_u32(ring);
    sbt_ptx::griddep_wait();
    const int j = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const Place at = place_of<V, INTER>(j, LPR, p.D, p.rot);
    const int kind = blockIdx.x >= p.blocks[0];
    const int32_t heads = p.heads[kind], hblocks = (heads + HB - 1) / HB;
    const char* const wp = p.w[kind];
    float w[2 * V], dw[2 * V];
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) w[e] = 1.f, dw[e] = 0.f;
    if (wp) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        unpack<KIND>(at.a >= 0 ? sbt_ld(reinterpret_cast<const uint4*>(wp + at.a * ES)) : zero, w);
        unpack<KIND>(at.b >= 0 ? sbt_ld(reinterpret_cast<const uint4*>(wp + at.b * ES)) : zero, w + V);
    }
    const float inv_d = 1.f / (float)p.D;
    const int64_t items = p.tokens * hblocks;
    const int64_t first = (int64_t)(kind ? blockIdx.x - p.blocks[0] : blockIdx.x) * GROUPS;
    const int64_t stride = (int64_t)p.blocks[kind] * GROUPS;
    const int64_t steps = first < items ? (items - first - 1) / stride + 1 : 0;
    const Item step = item_at(stride, hblocks);

    Item in = item_at(first + g, hblocks);  // the next item to load
    int32_t in_pos = in.t < p.tokens ? sbt_ld(p.pos + in.t) : -1;
    auto load = [&](int stage) {
        const uint32_t dst = ring_u32 + stage * VECS * kThreads * 16;
        if (in.t < p.tokens) {
            const int32_t h0 = in.hb * HB;
            const char* gr = p.g[kind].at(in.t, h0);
            const char* xr = p.x[kind].at(in.t, h0);
#pragma unroll
            for (int i = 0; i < HB; ++i)
                if (h0 + i < heads) {
                    const int64_t og = i * p.g[kind].ldh, ox = i * p.x[kind].ldh;
                    if (at.a >= 0) copy16(dst + (4 * i) * kThreads * 16, gr + og + at.a * ES);
                    if (at.b >= 0) copy16(dst + (4 * i + 1) * kThreads * 16, gr + og + at.b * ES);
                    if (wp && at.a >= 0) copy16(dst + (4 * i + 2) * kThreads * 16, xr + ox + at.a * ES);
                    if (wp && at.b >= 0) copy16(dst + (4 * i + 3) * kThreads * 16, xr + ox + at.b * ES);
                }
            if (in_pos >= 0 && in_pos < p.n_pos) {  // read only where something is turned
                const float2* row = p.table + (int64_t)in_pos * (p.rot / 2);
#pragma unroll
                for (int i = 0; i < AV; ++i) {
                    const int pair = at.pair[i / (AV / 2)];
                    if (pair >= 0) copy16_l1(dst + (4 * HB + i) * kThreads * 16, row + pair + 2 * (i % (AV / 2)));
                }
            }
        }
        copy_commit();
        s_pos[stage * kThreads] = in_pos;
        advance(in, step, hblocks);
        if (in.t < p.tokens) in_pos = sbt_ld(p.pos + in.t);
    };
#pragma unroll 1
    for (int s = 0; s < STAGES - 1; ++s) load(s);

    Item it = item_at(first + g, hblocks);
    int stage = 0;
#pragma unroll 1
    for (int64_t n = 0; n < steps; ++n) {
        copy_wait<STAGES - 2>();
        load(stage == 0 ? STAGES - 1 : stage - 1);
        const uint4* const v = ring + stage * VECS * kThreads;
        const bool on = it.t < p.tokens;
        const int32_t h0 = it.hb * HB, pos = s_pos[stage * kThreads];
        const bool real = on && pos >= 0 && (p.rot == 0 || pos < p.n_pos);
        const uint4 zero = make_uint4(0, 0, 0, 0), one = make_uint4(0x3F800000u, 0u, 0x3F800000u, 0u);
        float cs[V], sn[V];
#pragma unroll
        for (int i = 0; i < AV; ++i) {
            const uint4 c = real && at.pair[i / (AV / 2)] >= 0 ? v[(4 * HB + i) * kThreads] : one;
            cs[2 * i] = __uint_as_float(c.x), sn[2 * i] = __uint_as_float(c.y);
            cs[2 * i + 1] = __uint_as_float(c.z), sn[2 * i + 1] = __uint_as_float(c.w);
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            const bool row = on && h0 + i < heads;
            float u[2 * V];
            unpack<KIND>(row && real && at.a >= 0 ? v[(4 * i) * kThreads] : zero, u);
            unpack<KIND>(row && real && at.b >= 0 ? v[(4 * i + 1) * kThreads] : zero, u + V);
            turn<V, INTER>(u, at, cs, sn, -1.f);
            if (wp) {
                float x[2 * V], ss = 0.f, dot = 0.f;
                unpack<KIND>(row && real && at.a >= 0 ? v[(4 * i + 2) * kThreads] : zero, x);
                unpack<KIND>(row && real && at.b >= 0 ? v[(4 * i + 3) * kThreads] : zero, x + V);
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    ss += x[e] * x[e];
                    dot += u[e] * w[e] * x[e];
                }
                ss = lanes_sum<LPR>(ss);
                dot = lanes_sum<LPR>(dot);
                const float r = row && real ? rsqrtf(ss * inv_d + p.eps) : 0.f;
                const float c = dot * inv_d * r * r;
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    dw[e] += u[e] * (x[e] * r);  // nothing for rows of padding: u, x and r are zero
                    u[e] = r * (u[e] * w[e] - x[e] * c);
                }
            }
            if (row) {
                char* y = const_cast<char*>(p.dx[kind].at(it.t, h0 + i));
                if (at.a >= 0) *reinterpret_cast<uint4*>(y + at.a * ES) = pack<KIND>(u);
                if (at.b >= 0) *reinterpret_cast<uint4*>(y + at.b * ES) = pack<KIND>(u + V);
            }
        }
        advance(it, step, hblocks);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    copy_wait<0>();
    if (!wp) return;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) s_dw[(g * LPR + j) * 2 * V + e] = dw[e];
    __syncthreads();
    for (int c = threadIdx.x; c < LPR * 2 * V; c += kThreads) {
        const Place q = place_of<V, INTER>(c / (2 * V), LPR, p.D, p.rot);
        const int e = c % (2 * V), d = e < V ? q.a : q.b;
        if (d < 0) continue;
        float sum = 0.f;
        for (int i = 0; i < GROUPS; ++i) sum += s_dw[i * LPR * 2 * V + c];
        p.partial[(int64_t)blockIdx.x * p.D + d + e % V] = sum;
    }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) k_norm_rope_bwd_elems(const BwdParams p) {
    typedef typename Num<KIND>::T T;
    extern __shared__ float s_dw[];  // [warps][D]
    sbt_ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kind = blockIdx.x >= p.blocks[0];
    const int first = kind ? blockIdx.x - p.blocks[0] : blockIdx.x;
    const T* const w = reinterpret_cast<const T*>(p.w[kind]);
    const int64_t rows = p.tokens * p.heads[kind];
    float da[kMaxScalarPairs], db[kMaxScalarPairs];
#pragma unroll
    for (int i = 0; i < kMaxScalarPairs; ++i) da[i] = db[i] = 0.f;
    for (int64_t row = (int64_t)first * (kThreads / 32) + warp; row < rows;
         row += (int64_t)p.blocks[kind] * (kThreads / 32)) {
        const int64_t t = row / p.heads[kind];
        const int h = (int)(row - t * p.heads[kind]);
        const int32_t pos = sbt_ld(p.pos + t);
        const bool real = pos >= 0 && (p.rot == 0 || pos < p.n_pos);
        const T* gr = reinterpret_cast<const T*>(p.g[kind].at(t, h));
        const T* xr = w ? reinterpret_cast<const T*>(p.x[kind].at(t, h)) : nullptr;
        T* y = reinterpret_cast<T*>(const_cast<char*>(p.dx[kind].at(t, h)));
        float a[kMaxScalarPairs], b[kMaxScalarPairs], xa[kMaxScalarPairs], xb[kMaxScalarPairs], ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxScalarPairs; ++i) {
            const int pr = lane + 32 * i;
            int ia, ib;
            pair_at(pr, p.D, p.rot, p.interleaved, &ia, &ib);
            a[i] = ia >= 0 ? Num<KIND>::get(gr[ia]) : 0.f;
            b[i] = ib >= 0 ? Num<KIND>::get(gr[ib]) : 0.f;
            if (pr < p.rot / 2 && real) {
                const float2 cs = sbt_ld(p.table + (int64_t)pos * (p.rot / 2) + pr);
                const float u = a[i] * cs.x + b[i] * cs.y;
                b[i] = b[i] * cs.x - a[i] * cs.y;
                a[i] = u;
            }
            xa[i] = xb[i] = 0.f;
            if (w) {
                if (ia >= 0) {
                    xa[i] = Num<KIND>::get(xr[ia]);
                    ss += xa[i] * xa[i];
                    dot += a[i] * Num<KIND>::get(w[ia]) * xa[i];
                }
                if (ib >= 0) {
                    xb[i] = Num<KIND>::get(xr[ib]);
                    ss += xb[i] * xb[i];
                    dot += b[i] * Num<KIND>::get(w[ib]) * xb[i];
                }
            }
        }
        float r = 1.f, c = 0.f;
        if (w) {
            ss = lanes_sum<32>(ss);
            dot = lanes_sum<32>(dot);
            r = 1.f / sqrtf(ss / (float)p.D + p.eps);
            c = dot / (float)p.D * r * r;
        }
#pragma unroll
        for (int i = 0; i < kMaxScalarPairs; ++i) {
            int ia, ib;
            pair_at(lane + 32 * i, p.D, p.rot, p.interleaved, &ia, &ib);
            float u = a[i], v = b[i];
            if (w) {
                if (real) {
                    da[i] += u * (xa[i] * r);
                    db[i] += v * (xb[i] * r);
                }
                if (ia >= 0) u = r * (u * Num<KIND>::get(w[ia]) - xa[i] * c);
                if (ib >= 0) v = r * (v * Num<KIND>::get(w[ib]) - xb[i] * c);
            }
            if (ia >= 0) y[ia] = real ? Num<KIND>::put(u) : T(0);
            if (ib >= 0) y[ib] = real ? Num<KIND>::put(v) : T(0);
        }
    }
    if (!w) return;
#pragma unroll
    for (int i = 0; i < kMaxScalarPairs; ++i) {
        int ia, ib;
        pair_at(lane + 32 * i, p.D, p.rot, p.interleaved, &ia, &ib);
        if (ia >= 0) s_dw[warp * p.D + ia] = da[i];
        if (ib >= 0) s_dw[warp * p.D + ib] = db[i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
        float sum = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) sum += s_dw[i * p.D + d];
        p.partial[(int64_t)blockIdx.x * p.D + d] = sum;
    }
}

// dw[kind][d] = the blocks' sums: 128 strands of blocks side by side for eight
// elements, then the strands in a fixed order.
__global__ void __launch_bounds__(1024) k_norm_rope_dw(const BwdParams p) {
    __shared__ float s[32][8];
    sbt_ptx::griddep_wait();
    const int kind = blockIdx.y, c = threadIdx.x & 7, strand = threadIdx.x >> 3;
    const int d = blockIdx.x * 8 + c;
    if (!p.dw[kind]) return;
    const float* part = p.partial + (int64_t)(kind ? p.blocks[0] : 0) * p.D;
    float sum = 0.f;
    if (d < p.D)
#pragma unroll 4
        for (int i = strand; i < p.blocks[kind]; i += 128) sum += part[(int64_t)i * p.D + d];
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if ((threadIdx.x & 31) < 8) s[threadIdx.x >> 5][c] = sum;
    __syncthreads();
    if (threadIdx.x < 8 && d < p.D) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][c];
        p.dw[kind][d] = t;
    }
}

// -------------------------------------------------------------------------------- table

struct TableParams {
    float2* table;
    int64_t n_pos;
    int32_t rot;
    int32_t scaling;
    double base, factor, low, high, orig, amplitude;
};

// Angles are formed and reduced in 64 bits: at position 10^6 an fp32 product
// would already be off by 0.06.
__global__ void __launch_bounds__(kThreads) k_rope_table(const TableParams p) {
    sbt_ptx::griddep_wait();
    const int half = p.rot / 2;
    const int64_t n = p.n_pos * half;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t pos = i / half;
        const double e = -2.0 * (double)(i - pos * half) / (double)p.rot;
        double f = pow(p.base, e);
        if (p.scaling == SBT_ROPE_LINEAR) {
            f /= p.factor;
        } else if (p.scaling == SBT_ROPE_NTK) {
            f = p.rot > 2 ? pow(p.base * pow(p.factor, (double)p.rot / (double)(p.rot - 2)), e) : f;
        } else if (p.scaling == SBT_ROPE_BY_PARTS) {
            const double turns = p.orig * f / 6.283185307179586476925286766559;
            double keep = (turns - p.low) / (p.high - p.low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = (1.0 - keep) * f / p.factor + keep * f;
        }
        double s, c;
        sincos((double)pos * f, &s, &c);
        p.table[i] = make_float2((float)(c * p.amplitude), (float)(s * p.amplitude));
    }
}

int kind_of(sbt_dtype t) { return t == SBT_F32 ? kF32 : t == SBT_BF16 ? kBF16 : kF16; }

// Lanes per row of the vector path: every lane holds one pair of vectors.
int lanes_per_row(int D, int rot, int V, bool inter) {
    const int need = inter ? (D / V + 1) / 2 : rot / (2 * V) + ((D - rot) / V + 1) / 2;
    int l = 1;
    while (l < need) l *= 2;
    return l;
}

// Sizes the vector path takes (the caller checks the addresses).
bool sizes_ok(int D, int rot, int V, bool inter) {
    return D % V == 0 && (inter ? rot % V == 0 : rot % (2 * V) == 0) && lanes_per_row(D, rot, V, inter) <= 32;
}


// Splits `most` blocks over the kinds in proportion to their rows, none without
// work and none more than its items need.
template <int N>
void split_blocks(int64_t most, const int64_t (&need)[N], int32_t (&blocks)[N]) {
    int64_t total = 0, left = most;
    for (int i = 0; i < N; ++i) total += need[i];
    for (int i = N - 1; i >= 0; --i) {
        int64_t b = need[i];
        if (total > most) b = i ? std::max<int64_t>(1, most * need[i] / total) : left;
        blocks[i] = (int32_t)(need[i] ? std::min(b, need[i]) : 0);
        left -= blocks[i];
    }
}

template <int KIND, bool INTER, int LPR>
void fwd_launch(const sbt_context* ctx, const FwdParams& p, cudaStream_t stream) {
    constexpr int GROUPS = kThreads / LPR, HB = kFwdHeads;
    const int64_t total = p.heads[0] + p.heads[1] + p.heads[2];
    const unsigned ty = (unsigned)std::min<int64_t>(sbt_cdiv(p.tokens, GROUPS), 65535);
    const int64_t hb = sbt_cdiv(p.heads[0], HB) + sbt_cdiv(p.heads[1], HB) + sbt_cdiv(p.heads[2], HB);
    if (p.tokens * total >= (int64_t)ctx->sm_count * kManyRows * GROUPS && 3 * hb <= total)
        sbt_launch_dependent(k_norm_rope<KIND, INTER, LPR, HB>, dim3((unsigned)hb, ty), dim3(kThreads), 0, stream, p);
    else
        sbt_launch_dependent(k_norm_rope<KIND, INTER, LPR, 1>, dim3((unsigned)total, ty), dim3(kThreads), 0, stream, p);
}

template <int KIND, bool INTER, int LPR>
void bwd_launch(const sbt_context* ctx, const BwdParams& p, cudaStream_t stream) {
    constexpr int V = Num<KIND>::V;
    const size_t smem = std::max((size_t)kStages * kThreads * ((4 * kBwdHeads + V / 2) * 16 + 4),
                                 (size_t)kThreads * 2 * V * sizeof(float));
    constexpr auto kern = k_norm_rope_bwd<KIND, INTER, LPR, kBwdHeads, kStages>;
    sbt_resident_blocks<kern>(ctx, kThreads, smem);
    sbt_launch_dependent(kern, dim3(p.blocks[0] + p.blocks[1]), dim3(kThreads), smem, stream, p);
}

template <int KIND, bool INTER, class P, class F>
void by_lanes(int lpr, const P& p, F f) {
    switch (lpr) {
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        case 8: f(std::integral_constant<int, 8>()); break;
        case 16: f(std::integral_constant<int, 16>()); break;
        default: f(std::integral_constant<int, 32>()); break;
    }
}

template <int KIND>
void fwd(const sbt_context* ctx, const FwdParams& p, bool vec, cudaStream_t stream) {
    constexpr int V = Num<KIND>::V;
    if (!vec) {
        const int64_t rows = p.tokens * (p.heads[0] + p.heads[1] + p.heads[2]);
        const int64_t blocks = std::min<int64_t>(sbt_cdiv(rows, kThreads / 32), (int64_t)ctx->sm_count * 16);
        sbt_launch_dependent(k_norm_rope_elems<KIND>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
    } else if (p.interleaved) {
        by_lanes<KIND, true>(lanes_per_row(p.D, p.rot, V, true), p,
                             [&](auto n) { fwd_launch<KIND, true, decltype(n)::value>(ctx, p, stream); });
    } else {
        by_lanes<KIND, false>(lanes_per_row(p.D, p.rot, V, false), p,
                              [&](auto n) { fwd_launch<KIND, false, decltype(n)::value>(ctx, p, stream); });
    }
}

template <int KIND>
void bwd(const sbt_context* ctx, const BwdParams& p, bool vec, cudaStream_t stream) {
    constexpr int V = Num<KIND>::V;
    if (!vec) {
        sbt_launch_dependent(k_norm_rope_bwd_elems<KIND>, dim3(p.blocks[0] + p.blocks[1]), dim3(kThreads),
                             (kThreads / 32) * p.D * sizeof(float), stream, p);
    } else if (p.interleaved) {
        by_lanes<KIND, true>(lanes_per_row(p.D, p.rot, V, true), p,
                             [&](auto n) { bwd_launch<KIND, true, decltype(n)::value>(ctx, p, stream); });
    } else {
        by_lanes<KIND, false>(lanes_per_row(p.D, p.rot, V, false), p,
                              [&](auto n) { bwd_launch<KIND, false, decltype(n)::value>(ctx, p, stream); });
    }
}

bool rows_vec(const SbtHeadRows& r, int es) {
    return !r.p || (sbt_aligned16(r.p) && sbt_mul16(r.ld, es) && sbt_mul16(r.ldh, es));
}

Rows bytes_of(const SbtHeadRows& r, int es) { return Rows{(const char*)r.p, r.ld * es, r.ldh * es}; }

}  // namespace

sbt_status sbt_launch_norm_rope(sbt_context* ctx, sbt_dtype dtype, const SbtHeadRows& q, const SbtHeadRows& k,
                                const SbtHeadRows& v, const SbtHeadRows& q_out, const SbtHeadRows& k_out,
                                int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t D, const int32_t* pos,
                                const sbt_rope* rope, const void* wq, const void* wk, float eps,
                                const sbt_kv_cache* cache, const sbt_page_map* map, const int32_t* seq,
                                cudaStream_t stream) {
    const int es = sbt_dtype_size(dtype), V = 16 / es;
    FwdParams p = {};
    p.x[0] = bytes_of(q, es), p.x[1] = bytes_of(k, es), p.x[2] = bytes_of(v, es);
    p.y[0] = bytes_of(q_out, es), p.y[1] = bytes_of(k_out, es);
    p.w[0] = (const char*)wq, p.w[1] = (const char*)wk;
    p.heads[0] = q_heads, p.heads[1] = k_heads, p.heads[2] = cache && v.p ? k_heads : 0;
    p.tokens = tokens, p.D = D, p.pos = pos, p.eps = eps;
    if (rope && rope->rot_dim) {
        p.rot = rope->rot_dim, p.interleaved = rope->layout == SBT_ROPE_INTERLEAVED;
        p.table = (const float2*)rope->table, p.n_pos = rope->n_pos;
    }
    bool vec = ctx->path != SBT_PATH_SCALAR && sizes_ok(D, p.rot, V, p.interleaved) && rows_vec(q, es) &&
               rows_vec(k, es) && rows_vec(v, es) && rows_vec(q_out, es) && rows_vec(k_out, es) && sbt_aligned16(wq) &&
               sbt_aligned16(wk) && sbt_aligned16(p.table) && (p.rot / 2) % 2 == 0;
    if (cache) {
        p.cache[0] = (char*)cache->k, p.cache[1] = (char*)cache->v;
        p.ld_page = cache->ld_page * es, p.ld_slot = cache->ld_slot * es, p.ld_head = cache->ld_head * es;
        p.page_table = map->page_table, p.ld_table = map->ld_table, p.n_pages = map->n_pages;
        p.n_seq = map->n_seq, p.max_pages = map->max_pages, p.seq = seq;
        p.page_size = sbt_make_fastdiv((uint32_t)map->page_size);
        vec = vec && sbt_aligned16(cache->k) && sbt_aligned16(cache->v) && sbt_mul16(cache->ld_page, es) &&
              sbt_mul16(cache->ld_slot, es) && sbt_mul16(cache->ld_head, es);
    }
    switch (kind_of(dtype)) {
        case kF32: fwd<kF32>(ctx, p, vec, stream); break;
        case kBF16: fwd<kBF16>(ctx, p, vec, stream); break;
        default: fwd<kF16>(ctx, p, vec, stream); break;
    }
    return sbt_after_launch(ctx, "qk_norm_rope");
}

int sbt_norm_rope_bwd_blocks(const sbt_context* ctx) { return ctx->sm_count * 4; }

sbt_status sbt_launch_norm_rope_bwd(sbt_context* ctx, sbt_dtype dtype, const SbtHeadRows& gq, const SbtHeadRows& gk,
                                    const SbtHeadRows& q, const SbtHeadRows& k, const SbtHeadRows& dq,
                                    const SbtHeadRows& dk, int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t D,
                                    const int32_t* pos, const sbt_rope* rope, const void* wq, const void* wk,
                                    float eps, float* dwq, float* dwk, void* workspace, cudaStream_t stream) {
    const int es = sbt_dtype_size(dtype), V = 16 / es;
    BwdParams p = {};
    p.g[0] = bytes_of(gq, es), p.g[1] = bytes_of(gk, es);
    p.x[0] = bytes_of(q, es), p.x[1] = bytes_of(k, es);
    p.dx[0] = bytes_of(dq, es), p.dx[1] = bytes_of(dk, es);
    p.w[0] = (const char*)wq, p.w[1] = (const char*)wk;
    p.heads[0] = q_heads, p.heads[1] = k_heads;
    p.tokens = tokens, p.D = D, p.pos = pos, p.eps = eps;
    if (rope && rope->rot_dim) {
        p.rot = rope->rot_dim, p.interleaved = rope->layout == SBT_ROPE_INTERLEAVED;
        p.table = (const float2*)rope->table, p.n_pos = rope->n_pos;
    }
    p.partial = (float*)workspace;
    p.dw[0] = dwq, p.dw[1] = dwk;
    const bool vec = ctx->path != SBT_PATH_SCALAR && sizes_ok(D, p.rot, V, p.interleaved) && rows_vec(gq, es) &&
                     rows_vec(gk, es) && rows_vec(q, es) && rows_vec(k, es) && rows_vec(dq, es) && rows_vec(dk, es) &&
                     sbt_aligned16(wq) && sbt_aligned16(wk) && sbt_aligned16(p.table) && (p.rot / 2) % 2 == 0;
    // blocks in proportion to the head rows, none without work
    const int lpr = vec ? lanes_per_row(D, p.rot, V, p.interleaved) : 32;
    const int64_t groups = kThreads / lpr, hb = vec ? kBwdHeads : 1;
    const int64_t need[2] = {sbt_cdiv(tokens * sbt_cdiv(q_heads, hb), groups),
                             sbt_cdiv(tokens * sbt_cdiv(k_heads, hb), groups)};
    split_blocks(sbt_norm_rope_bwd_blocks(ctx), need, p.blocks);
    sbt_status st = SBT_OK;
    if (p.blocks[0] + p.blocks[1] > 0) {  // no rows: only the weights' gradients, which are zero
        switch (kind_of(dtype)) {
            case kF32: bwd<kF32>(ctx, p, vec, stream); break;
            case kBF16: bwd<kBF16>(ctx, p, vec, stream); break;
            default: bwd<kF16>(ctx, p, vec, stream); break;
        }
        st = sbt_after_launch(ctx, "qk_norm_rope_backward");
    }
    if (st || (!dwq && !dwk)) return st;
    if ((st = sbt_cuda_check(sbt_launch_dependent(k_norm_rope_dw, dim3((D + 7) / 8, 2), dim3(1024), 0, stream, p),
                             "qk_norm_rope_backward sums launch")))
        return st;
    return sbt_after_launch(ctx, "qk_norm_rope_backward sums");
}

sbt_status sbt_launch_rope_table(sbt_context* ctx, float* table, int64_t n_pos, int32_t rot, double base, int scaling,
                                 double factor, int64_t orig, double low, double high, double amplitude,
                                 cudaStream_t stream) {
    TableParams p = {(float2*)table, n_pos, rot, scaling, base, factor, low, high, (double)orig, amplitude};
    const int64_t blocks = std::min<int64_t>(sbt_cdiv(n_pos * (rot / 2), kThreads), (int64_t)ctx->sm_count * 16);
    sbt_launch_dependent(k_rope_table, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
    return sbt_after_launch(ctx, "rope_table");
}
