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
#include <type_traits>

#include "sbt_internal.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kThreads = 256;
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
    if (Num<KIND>::V == 4) {
        x[0] = Num<KIND>::get((typename Num<KIND>::T)v.x), x[1] = Num<KIND>::get((typename Num<KIND>::T)v.y);
        x[2] = Num<KIND>::get((typename Num<KIND>::T)v.z), x[3] = Num<KIND>::get((typename Num<KIND>::T)v.w);
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[(2 * i) % Num<KIND>::V] = Num<KIND>::get((typename Num<KIND>::T)(w[i] & 0xFFFFu));
            x[(2 * i + 1) % Num<KIND>::V] = Num<KIND>::get((typename Num<KIND>::T)(w[i] >> 16));
        }
    }
}

template <int KIND>
__device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = Num<KIND>::V == 4 ? (uint32_t)Num<KIND>::put(x[i % Num<KIND>::V])
                                 : (uint32_t)Num<KIND>::put(x[(2 * i) % Num<KIND>::V]) |
                                       (uint32_t)Num<KIND>::put(x[(2 * i + 1) % Num<KIND>::V]) << 16;
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
    const int64_t s = p.seq ? (int64_t)__ldg(p.seq + t) : t;
    if (s < 0 || s >= p.n_seq || pos < 0) return -1;
    const uint32_t j = sbt_div(p.page_size, (uint32_t)pos);
    if (j >= (uint32_t)p.max_pages) return -1;
    const int32_t page = __ldg(p.page_table + s * p.ld_table + j);
    if (page < 0 || page >= p.n_pages) return -1;
    return page * p.ld_page + (int64_t)(pos - (int32_t)(j * p.page_size.d)) * p.ld_slot;
}

// The two vectors of lane j of a row: element offsets (-1: none) and the pair
// the first of them starts with in the table (-1: not turned).
struct Place {
    int a, b, pair;
};
template <int V, bool INTER>
__device__ __forceinline__ Place place_of(int j, int D, int rot) {
    Place q;
    if (INTER) {
        q.a = 2 * j * V < D ? 2 * j * V : -1;
        q.b = (2 * j + 1) * V < D ? (2 * j + 1) * V : -1;
        q.pair = q.a >= 0 && q.a < rot ? q.a / 2 : -1;
        return q;
    }
    const int np = rot / (2 * V);
    if (j < np) {
        q.a = j * V;
        q.b = rot / 2 + j * V;
        q.pair = j * V;
    } else {
        const int d = rot + 2 * (j - np) * V;
        q.a = d < D ? d : -1;
        q.b = d + V < D ? d + V : -1;
        q.pair = -1;
    }
    return q;
}

// cos and sin of this lane's V pairs.
template <int V, bool INTER>
__device__ __forceinline__ void angles(const float2* row, const Place& q, int rot, float* cs, float* sn) {
#pragma unroll
    for (int i = 0; i < V; ++i) cs[i] = 1.f, sn[i] = 0.f;
    if (q.pair < 0) return;
    // interleaved: a vector holds V / 2 pairs, and the second vector may lie past rot_dim
    const int n = INTER && (q.b < 0 || q.b >= rot) ? V / 2 : V;
#pragma unroll
    for (int i = 0; i < V; i += 2)
        if (i < n) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(row + q.pair + i));
            cs[i] = c.x, sn[i] = c.y, cs[i + 1] = c.z, sn[i + 1] = c.w;
        }
}

// Turns the lane's 2 V elements (x[0..V) of vector a, x[V..2V) of vector b); sign -1: the transpose.
template <int V, bool INTER>
__device__ __forceinline__ void turn(float* x, const float* cs, const float* sn, float sign) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
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

// HB heads per group: grid (head blocks, token blocks).
template <int KIND, bool INTER, int LPR, int HB>
__global__ void __launch_bounds__(kThreads) k_norm_rope(const FwdParams p) {
    constexpr int V = Num<KIND>::V, ES = 16 / V, GROUPS = kThreads / LPR;
    const int j = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const Place at = place_of<V, INTER>(j, p.D, p.rot);
    const int total = p.heads[0] + p.heads[1] + p.heads[2];
    const int h0 = blockIdx.x * HB;
    for (int64_t t0 = (int64_t)blockIdx.y * GROUPS; t0 < p.tokens; t0 += (int64_t)gridDim.y * GROUPS) {
        const int64_t t = t0 + g;
        const bool on = t < p.tokens;
        uint4 va[HB], vb[HB];
        int kind[HB], head[HB];
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            int h = h0 + i;
            kind[i] = h >= total ? -1 : h < p.heads[0] ? 0 : h < p.heads[0] + p.heads[1] ? 1 : 2;
            head[i] = h - (kind[i] >= 1 ? p.heads[0] : 0) - (kind[i] == 2 ? p.heads[1] : 0);
            va[i] = vb[i] = make_uint4(0, 0, 0, 0);
            if (kind[i] >= 0 && on) {
                const char* x = p.x[kind[i]].at(t, head[i]);
                if (at.a >= 0) va[i] = *reinterpret_cast<const uint4*>(x + at.a * ES);
                if (at.b >= 0) vb[i] = *reinterpret_cast<const uint4*>(x + at.b * ES);
            }
        }
        const int32_t pos = on ? __ldg(p.pos + t) : -1;
        const bool real = pos >= 0 && (p.rot == 0 || pos < p.n_pos);
        int64_t slot = -1;
        if (p.cache[0] && h0 + HB > p.heads[0] && real) slot = cache_slot(p, t, pos);
        float cs[V], sn[V];
        if (p.rot && real) {
            angles<V, INTER>(p.table + (int64_t)pos * (p.rot / 2), at, p.rot, cs, sn);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) cs[i] = 1.f, sn[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (kind[i] < 0) break;  // the same for the whole block
            if (kind[i] < 2) {
                float x[2 * V];
                unpack<KIND>(va[i], x);
                unpack<KIND>(vb[i], x + V);
                if (p.w[kind[i]]) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) ss += x[e] * x[e];
                    const float r = 1.f / sqrtf(lanes_sum<LPR>(ss) / (float)p.D + p.eps);
                    float w[2 * V];
                    const uint4 one = make_uint4(0, 0, 0, 0);
                    unpack<KIND>(at.a >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.w[kind[i]] + at.a * ES)) : one, w);
                    unpack<KIND>(at.b >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.w[kind[i]] + at.b * ES)) : one, w + V);
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) x[e] = x[e] * r * w[e];
                }
                turn<V, INTER>(x, cs, sn, 1.f);
                va[i] = real ? pack<KIND>(x) : make_uint4(0, 0, 0, 0);
                vb[i] = real ? pack<KIND>(x + V) : make_uint4(0, 0, 0, 0);
                if (p.y[kind[i]].p && on) {
                    char* y = const_cast<char*>(p.y[kind[i]].at(t, head[i]));
                    if (at.a >= 0) *reinterpret_cast<uint4*>(y + at.a * ES) = va[i];
                    if (at.b >= 0) *reinterpret_cast<uint4*>(y + at.b * ES) = vb[i];
                }
            }
            if (kind[i] >= 1 && slot >= 0) {
                char* y = p.cache[kind[i] - 1] + slot + head[i] * p.ld_head;
                if (at.a >= 0) *reinterpret_cast<uint4*>(y + at.a * ES) = va[i];
                if (at.b >= 0) *reinterpret_cast<uint4*>(y + at.b * ES) = vb[i];
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
    const int lane = threadIdx.x & 31;
    const int total = p.heads[0] + p.heads[1] + p.heads[2];
    const int64_t rows = p.tokens * total;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); row < rows;
         row += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t t = row / total;
        int h = (int)(row - t * total);
        const int kind = h < p.heads[0] ? 0 : h < p.heads[0] + p.heads[1] ? 1 : 2;
        h -= (kind >= 1 ? p.heads[0] : 0) + (kind == 2 ? p.heads[1] : 0);
        const int32_t pos = __ldg(p.pos + t);
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
                const float2 cs = __ldg(p.table + (int64_t)pos * (p.rot / 2) + pr);
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

// One block takes head rows of the queries or of the keys only, so one set of
// sums for dw stays in registers; the blocks' sums go to the workspace and are
// added in block order by k_norm_rope_dw: no atomics, the same bits every run.
template <int KIND, bool INTER, int LPR, int HB>
__global__ void __launch_bounds__(kThreads) k_norm_rope_bwd(const BwdParams p) {
    constexpr int V = Num<KIND>::V, ES = 16 / V, GROUPS = kThreads / LPR;
    extern __shared__ float s_dw[];  // [GROUPS][LPR * 2 V]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int j = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const Place at = place_of<V, INTER>(j, p.D, p.rot);
    const int kind = blockIdx.x >= p.blocks[0];
    const int first = kind ? blockIdx.x - p.blocks[0] : blockIdx.x;
    const int heads = p.heads[kind], hblocks = (heads + HB - 1) / HB;
    const char* const wp = p.w[kind];
    float w[2 * V], dw[2 * V];
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) w[e] = 1.f, dw[e] = 0.f;
    if (wp) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        unpack<KIND>(at.a >= 0 ? __ldg(reinterpret_cast<const uint4*>(wp + at.a * ES)) : zero, w);
        unpack<KIND>(at.b >= 0 ? __ldg(reinterpret_cast<const uint4*>(wp + at.b * ES)) : zero, w + V);
    }
    // items: (token, head block), tokens slowest
    const int64_t items = p.tokens * hblocks;
    for (int64_t i0 = (int64_t)first * GROUPS; i0 < items; i0 += (int64_t)p.blocks[kind] * GROUPS) {
        const int64_t it = i0 + g;
        const bool on = it < items;
        const int64_t t = on ? it / hblocks : 0;
        const int h0 = on ? (int)(it - t * hblocks) * HB : 0;
        uint4 ga[HB], gb[HB], xa[HB], xb[HB];
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            ga[i] = gb[i] = xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
            if (on && h0 + i < heads) {
                const char* gr = p.g[kind].at(t, h0 + i);
                if (at.a >= 0) ga[i] = *reinterpret_cast<const uint4*>(gr + at.a * ES);
                if (at.b >= 0) gb[i] = *reinterpret_cast<const uint4*>(gr + at.b * ES);
                if (wp) {
                    const char* xr = p.x[kind].at(t, h0 + i);
                    if (at.a >= 0) xa[i] = *reinterpret_cast<const uint4*>(xr + at.a * ES);
                    if (at.b >= 0) xb[i] = *reinterpret_cast<const uint4*>(xr + at.b * ES);
                }
            }
        }
        const int32_t pos = on ? __ldg(p.pos + t) : -1;
        const bool real = pos >= 0 && (p.rot == 0 || pos < p.n_pos);
        float cs[V], sn[V];
        if (p.rot && real) {
            angles<V, INTER>(p.table + (int64_t)pos * (p.rot / 2), at, p.rot, cs, sn);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) cs[i] = 1.f, sn[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            float u[2 * V];
            unpack<KIND>(ga[i], u);
            unpack<KIND>(gb[i], u + V);
            turn<V, INTER>(u, cs, sn, -1.f);
            if (wp) {
                float x[2 * V], ss = 0.f, dot = 0.f;
                unpack<KIND>(xa[i], x);
                unpack<KIND>(xb[i], x + V);
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    ss += x[e] * x[e];
                    dot += u[e] * w[e] * x[e];
                }
                ss = lanes_sum<LPR>(ss);
                dot = lanes_sum<LPR>(dot);
                const float r = 1.f / sqrtf(ss / (float)p.D + p.eps);
                const float c = dot / (float)p.D * r * r;
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    if (real) dw[e] += u[e] * (x[e] * r);
                    u[e] = r * (u[e] * w[e] - x[e] * c);
                }
            }
            if (on && h0 + i < heads) {
                char* y = const_cast<char*>(p.dx[kind].at(t, h0 + i));
                const uint4 zero = make_uint4(0, 0, 0, 0);
                if (at.a >= 0) *reinterpret_cast<uint4*>(y + at.a * ES) = real ? pack<KIND>(u) : zero;
                if (at.b >= 0) *reinterpret_cast<uint4*>(y + at.b * ES) = real ? pack<KIND>(u + V) : zero;
            }
        }
    }
    if (!wp) return;
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) s_dw[(g * LPR + j) * 2 * V + e] = dw[e];
    __syncthreads();
    for (int c = threadIdx.x; c < LPR * 2 * V; c += kThreads) {
        const Place q = place_of<V, INTER>(c / (2 * V), p.D, p.rot);
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
        const int32_t pos = __ldg(p.pos + t);
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
                const float2 cs = __ldg(p.table + (int64_t)pos * (p.rot / 2) + pr);
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

// dw[kind][d] = the blocks' sums, in block order within each of 32 strands and then over the strands.
__global__ void __launch_bounds__(1024) k_norm_rope_dw(const BwdParams p) {
    __shared__ float s[32][33];
    sbt_ptx::griddep_wait();
    const int kind = blockIdx.y, c = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + c;
    if (!p.dw[kind]) return;
    const float* part = p.partial + (int64_t)(kind ? p.blocks[0] : 0) * p.D;
    float sum = 0.f;
    if (d < p.D)
#pragma unroll 4
        for (int i = strand; i < p.blocks[kind]; i += 32) sum += part[(int64_t)i * p.D + d];
    s[strand][c] = sum;
    __syncthreads();
    if (strand == 0 && d < p.D) {
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

template <int KIND, bool INTER, int LPR>
void fwd_launch(const FwdParams& p, int sms, cudaStream_t stream) {
    constexpr int GROUPS = kThreads / LPR;
    const int total = p.heads[0] + p.heads[1] + p.heads[2];
    int64_t ty = sbt_cdiv(p.tokens, GROUPS);
    if (ty > 65535) ty = 65535;
    // Four heads per group once that leaves two blocks for every SM; one head per group below.
    if (ty * sbt_cdiv(total, 4) >= 2 * sms)
        k_norm_rope<KIND, INTER, LPR, 4><<<dim3((unsigned)sbt_cdiv(total, 4), (unsigned)ty), kThreads, 0, stream>>>(p);
    else
        k_norm_rope<KIND, INTER, LPR, 1><<<dim3((unsigned)total, (unsigned)ty), kThreads, 0, stream>>>(p);
}

template <int KIND, bool INTER, int LPR>
void bwd_launch(const BwdParams& p, cudaStream_t stream) {
    const size_t smem = (size_t)kThreads * 2 * Num<KIND>::V * sizeof(float);
    k_norm_rope_bwd<KIND, INTER, LPR, 2><<<p.blocks[0] + p.blocks[1], kThreads, smem, stream>>>(p);
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
void fwd(const FwdParams& p, bool vec, int sms, cudaStream_t stream) {
    constexpr int V = Num<KIND>::V;
    if (!vec) {
        const int64_t rows = p.tokens * (p.heads[0] + p.heads[1] + p.heads[2]);
        const int64_t blocks = std::min<int64_t>(sbt_cdiv(rows, kThreads / 32), (int64_t)sms * 16);
        k_norm_rope_elems<KIND><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    } else if (p.interleaved) {
        by_lanes<KIND, true>(lanes_per_row(p.D, p.rot, V, true), p,
                             [&](auto n) { fwd_launch<KIND, true, decltype(n)::value>(p, sms, stream); });
    } else {
        by_lanes<KIND, false>(lanes_per_row(p.D, p.rot, V, false), p,
                              [&](auto n) { fwd_launch<KIND, false, decltype(n)::value>(p, sms, stream); });
    }
}

template <int KIND>
void bwd(const BwdParams& p, bool vec, cudaStream_t stream) {
    constexpr int V = Num<KIND>::V;
    if (!vec) {
        k_norm_rope_bwd_elems<KIND><<<p.blocks[0] + p.blocks[1], kThreads, (kThreads / 32) * p.D * sizeof(float),
                                      stream>>>(p);
    } else if (p.interleaved) {
        by_lanes<KIND, true>(lanes_per_row(p.D, p.rot, V, true), p,
                             [&](auto n) { bwd_launch<KIND, true, decltype(n)::value>(p, stream); });
    } else {
        by_lanes<KIND, false>(lanes_per_row(p.D, p.rot, V, false), p,
                              [&](auto n) { bwd_launch<KIND, false, decltype(n)::value>(p, stream); });
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
        case kF32: fwd<kF32>(p, vec, ctx->sm_count, stream); break;
        case kBF16: fwd<kBF16>(p, vec, ctx->sm_count, stream); break;
        default: fwd<kF16>(p, vec, ctx->sm_count, stream); break;
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
    const int64_t groups = kThreads / lpr, hb = vec ? 2 : 1;
    const int64_t need_q = sbt_cdiv(tokens * sbt_cdiv(q_heads, hb), groups);
    const int64_t need_k = sbt_cdiv(tokens * sbt_cdiv(k_heads, hb), groups);
    const int64_t most = sbt_norm_rope_bwd_blocks(ctx);
    int64_t bq = need_q, bk = need_k;
    if (bq + bk > most) {
        bk = k_heads ? std::max<int64_t>(1, most * k_heads / (q_heads + k_heads)) : 0;
        bk = std::min(bk, need_k);
        bq = q_heads ? std::min(need_q, most - bk) : 0;
    }
    p.blocks[0] = (int32_t)bq, p.blocks[1] = (int32_t)bk;
    sbt_status st = SBT_OK;
    if (bq + bk > 0) {  // no rows: only the weights' gradients, which are zero
        switch (kind_of(dtype)) {
            case kF32: bwd<kF32>(p, vec, stream); break;
            case kBF16: bwd<kBF16>(p, vec, stream); break;
            default: bwd<kF16>(p, vec, stream); break;
        }
        st = sbt_after_launch(ctx, "qk_norm_rope_backward");
    }
    if (st || (!dwq && !dwk)) return st;
    if ((st = sbt_cuda_check(sbt_launch_dependent(k_norm_rope_dw, dim3((D + 31) / 32, 2), dim3(1024), 0, stream, p),
                             "qk_norm_rope_backward sums launch")))
        return st;
    return sbt_after_launch(ctx, "qk_norm_rope_backward sums");
}

sbt_status sbt_launch_rope_table(sbt_context* ctx, float* table, int64_t n_pos, int32_t rot, double base, int scaling,
                                 double factor, int64_t orig, double low, double high, double amplitude,
                                 cudaStream_t stream) {
    TableParams p = {(float2*)table, n_pos, rot, scaling, base, factor, low, high, (double)orig, amplitude};
    const int64_t blocks = std::min<int64_t>(sbt_cdiv(n_pos * (rot / 2), kThreads), (int64_t)ctx->sm_count * 16);
    k_rope_table<<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    return sbt_after_launch(ctx, "rope_table");
}
