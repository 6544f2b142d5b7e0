// Root-mean-square norm of rows with the residual's addition, its output as
// numbers or as 8-bit codes with a power-of-two scale per block, and the
// gradient.
//
// Forward, for one row of C columns, in fp32:
//   h = x + r,   y = h w / sqrt(mean(h^2) + eps);
// h and y are rounded once each, at their stores (the norm takes the unrounded
// h).  Codes of a block of columns: with e the least integer for which no |y| of
// the block passes largest * 2^e, the codes are y 2^-e to nearest even and the
// scale is 2^e, so no code saturates and each is within half a step of y.
// Backward, with s = 1 / sqrt(mean(h^2) + eps) and g = w gy:
//   dx = gh + s (g - h s^2 mean(g h)),   dw = sum over rows of gy h s.
//
// Memory bounds both (about one flop a byte): a row is read once into registers
// and written once.  A row belongs to a power-of-two number of threads, a warp
// to 1024, which hold it in units of eight neighbouring elements (one 16-byte
// vector; two in fp32) or, where widths or addresses do not allow vectors, of
// one element.  Rows that start anywhere, but those of all arrays at the same place
// relative to 16 bytes, have vectors all the same (SHIFT).  Rows too wide for
// that, and codes without vectors, are read twice by k_add_norm_any and
// k_add_norm_bwd_any.
//
// Measured (GB300; at the copy rate in brackets): 16384 x 8192 bf16 with the
// residual to codes 162 us (139), to numbers 152 (119); 16384 x 4096 fp32 157 (119);
// 333 x 5003 fp16 6.9 us (2.0), element by element 7.2; a single row 5.4, what the
// host takes for a call (2.0 in a graph).  Gradient, 16384 x 4096 bf16 89 us (79), of
// which the second launch (the blocks' sums for dw) is 4; 1021 x 1537 fp32 8.6 (3.7).
// The forms that read twice, element by element, bf16: 4096 x 20480 252 us (99),
// gradient of 8192 x 16384 665 (159), of 16384 x 4097 340 (79).
#include <algorithm>

#include "sbt_internal.cuh"
#include "sbt_num.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace sbt_num;
using sbt_ptx::griddep_wait;

constexpr int kAnyThreads = 256;
constexpr int kLeastScale = -124;  // least exponent of a scale: products of scaled codes stay normal numbers

// W neighbouring elements as they lie in memory.
template <int KIND, int W> struct Unit;
template <int KIND> struct Unit<KIND, 8> {
    static constexpr int N = KIND == kF32 ? 2 : 1;
    uint4 v[N];
    __device__ __forceinline__ void load(const void* p) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = sbt_ld(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float* x) const {
#pragma unroll
        for (int i = 0; i < N; ++i) unpack<KIND>(v[i], x + 4 * i);
    }
    static __device__ __forceinline__ void store(void* p, const float* x) {
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p)[i] = pack<KIND>(x + 4 * i);
    }
};
template <int KIND> struct Unit<KIND, 1> {
    typedef typename Num<KIND>::T T;
    T v;
    __device__ __forceinline__ void load(const void* p) { v = sbt_ld(reinterpret_cast<const T*>(p)); }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void get(float* x) const { x[0] = Num<KIND>::get(v); }
    static __device__ __forceinline__ void store(void* p, const float* x) {
        *reinterpret_cast<T*>(p) = Num<KIND>::put(x[0]);
    }
};

struct NormParams {
    const char *x, *r, *w;      // r, w may be NULL
    char *h, *y;                // may be NULL
    int64_t ld_x, ld_r, ld_h, ld_y, ld_codes, ld_scales;  // bytes
    uint8_t *codes, *scales;    // NULL: none
    int64_t rows;
    int32_t cols, group, block, e5m2;
    float eps;
};

// Sums over the G threads of a row: one warp, or the whole block.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int G, float (*s)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int d = 16; d; d >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
    if (G == 32) return;
    const int lane = threadIdx.x & 31, warps = G >> 5;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) s[threadIdx.x >> 5][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = lane < warps ? s[lane][k] : 0.f;
#pragma unroll
        for (int d = 16; d; d >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
    }
}

// Biased exponent of the scale of a block whose largest |y| is `top` (255: NaN,
// for a block that holds an infinity or NaN).  448 and 57344 are 1.75 times a
// power of two.
__device__ __forceinline__ int scale_code(float top, int e5m2) {
    const uint32_t b = __float_as_uint(top);
    if (b == 0) return 127;
    if (b >= 0x7f800000u) return 255;
    const int e = (int)(b >> 23) - (e5m2 ? 15 : 8) + ((b & 0x7fffffu) > 0x600000u);
    return max(e, 127 + kLeastScale);
}

// 2^-e of a scale's code; NaN for 255, which makes the block's codes NaN.
__device__ __forceinline__ float scale_inverse(int code) {
    return code == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(254 - code) << 23);
}

// Two codes, to nearest even; `lo` in the low byte.
__device__ __forceinline__ uint32_t codes_of(float lo, float hi, int e5m2) {
    uint16_t c;
    if (e5m2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}

// The larger of two magnitudes, NaN if either is (their bits order them).
__device__ __forceinline__ float larger(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// SHIFT: rows that start anywhere, but all arrays' at the same place relative to 16 bytes.  Units are counted from the
// boundary before the row, so that all but its first and last are vectors; the weights are read element by element.
template <int KIND, int W, int NV, bool CODES, bool SHIFT>
__global__ void __launch_bounds__(W * NV == 32 ? 512 : 1024) k_add_norm(const NormParams p) {
    typedef Unit<KIND, W> U;
    typedef typename Num<KIND>::T T;
    constexpr int ES = sizeof(T), B = W * ES;
    // weights before the sum where registers allow, under it (from L2) otherwise: 16384 x 8192 bf16 to codes 202 and 161 us
    constexpr bool EARLY = !SHIFT && W * NV < 32;
    __shared__ float s_sum[32][1];
    griddep_wait();
    const int G = p.group, j = threadIdx.x & (G - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
    if (row >= p.rows) return;  // whole warps: a block of several rows has a warp for each
    const int phase = SHIFT ? (int)((reinterpret_cast<uintptr_t>(p.x + row * p.ld_x) & (B - 1)) / ES) : 0;
    const int units = SHIFT ? (p.cols + phase + W - 1) / W : p.cols / W;
    // unit u of an array's row; in the first and the last of a shifted row the elements that there are
    auto load = [&](U& x, const char* at, int u) {
        const int e = u * W - phase;
        if (!SHIFT || (e >= 0 && e + W <= p.cols)) {
            x.load(at + (int64_t)e * ES);
        } else {
            x.zero();
            for (int k = 0; k < W; ++k)
                if (e + k >= 0 && e + k < p.cols) reinterpret_cast<T*>(&x)[k] = sbt_ld(reinterpret_cast<const T*>(at) + e + k);
        }
    };
    auto store = [&](char* at, int u, const float* x) {
        const int e = u * W - phase;
        if (!SHIFT || (e >= 0 && e + W <= p.cols)) {
            U::store(at + (int64_t)e * ES, x);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (e + k >= 0 && e + k < p.cols) reinterpret_cast<T*>(at)[e + k] = Num<KIND>::put(x[k]);
        }
    };
    auto weights = [&](float (&t)[W], int u) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int e = u * W - phase + k;
            t[k] = e >= 0 && e < p.cols ? Num<KIND>::get(sbt_ld(reinterpret_cast<const T*>(p.w) + e)) : 0.f;
        }
    };
    U a[NV], b[NV], w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = j + i * G;
        a[i].zero(), b[i].zero();
        if (u < units) {
            load(a[i], p.x + row * p.ld_x, u);
            if (p.r) load(b[i], p.r + row * p.ld_r, u);
            if (EARLY && p.w) w[i].load(p.w + (int64_t)u * B);
        }
    }
    float h[NV][W], sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float t[W];
        a[i].get(h[i]);
        if (p.r) {
            b[i].get(t);
#pragma unroll
            for (int k = 0; k < W; ++k) h[i][k] += t[k];
        }
#pragma unroll
        for (int k = 0; k < W; ++k) sum[0] += h[i][k] * h[i][k];
    }
    if (!EARLY && !SHIFT && p.w)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (j + i * G < units) w[i].load(p.w + (int64_t)(j + i * G) * B);
    row_sums(sum, G, s_sum);
    const float s = 1.f / sqrtf(sum[0] / (float)p.cols + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = j + i * G;
        const bool ok = u < units;
        if (ok && p.h) store(p.h + row * p.ld_h, u, h[i]);
        if (p.w) {
            float t[W];
            if constexpr (SHIFT)
                weights(t, u);
            else
                w[i].get(t);
#pragma unroll
            for (int k = 0; k < W; ++k) h[i][k] = h[i][k] * s * t[k];
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) h[i][k] *= s;
        }
        if (ok && p.y) store(p.y + row * p.ld_y, u, h[i]);
        if constexpr (CODES) {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) top = larger(top, fabsf(h[i][k]));
            if (!ok) top = 0.f;
            for (int d = 1; d < p.block / W; d <<= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, d));
            const int code = scale_code(top, p.e5m2);
            const float inv = scale_inverse(code);
            uint32_t c[W / 4];
#pragma unroll
            for (int k = 0; k < W / 4; ++k)
                c[k] = codes_of(h[i][4 * k] * inv, h[i][4 * k + 1] * inv, p.e5m2) |
                       codes_of(h[i][4 * k + 2] * inv, h[i][4 * k + 3] * inv, p.e5m2) << 16;
            if (ok) {
                *reinterpret_cast<uint2*>(p.codes + row * p.ld_codes + (int64_t)u * W) = make_uint2(c[0], c[1]);
                const int per = p.block / W;
                if ((u & (per - 1)) == 0) p.scales[row * p.ld_scales + u / per] = (uint8_t)code;
            }
        }
    }
}

// Any width, stride and address: a block reads a row for its sum and again for
// its output; with codes a warp takes a scale's block of columns at a time.
template <int KIND>
__global__ void __launch_bounds__(kAnyThreads) k_add_norm_any(const NormParams p) {
    typedef typename Num<KIND>::T T;
    __shared__ float s_sum[32][1];
    griddep_wait();
    const int64_t row = blockIdx.x;
    const T* const x = reinterpret_cast<const T*>(p.x + row * p.ld_x);
    const T* const r = p.r ? reinterpret_cast<const T*>(p.r + row * p.ld_r) : nullptr;
    const T* const w = reinterpret_cast<const T*>(p.w);
    T* const h_out = p.h ? reinterpret_cast<T*>(p.h + row * p.ld_h) : nullptr;
    T* const y_out = p.y ? reinterpret_cast<T*>(p.y + row * p.ld_y) : nullptr;
    auto sum_at = [&](int c) { return Num<KIND>::get(sbt_ld(x + c)) + (r ? Num<KIND>::get(sbt_ld(r + c)) : 0.f); };
    float sum[1] = {0.f};
#pragma unroll 4
    for (int c = threadIdx.x; c < p.cols; c += kAnyThreads) {
        const float h = sum_at(c);
        sum[0] += h * h;
    }
    row_sums(sum, kAnyThreads, s_sum);
    const float s = 1.f / sqrtf(sum[0] / (float)p.cols + p.eps);
    auto out_at = [&](int c) {
        const float h = sum_at(c), y = h * s * (w ? Num<KIND>::get(sbt_ld(w + c)) : 1.f);
        if (h_out) h_out[c] = Num<KIND>::put(h);
        if (y_out) y_out[c] = Num<KIND>::put(y);
        return y;
    };
    if (!p.codes) {
#pragma unroll 4
        for (int c = threadIdx.x; c < p.cols; c += kAnyThreads) out_at(c);
        return;
    }
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < p.cols / p.block; b += kAnyThreads / 32) {
        float y[4], top = 0.f;  // a block has 128 columns at most
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = i * 32 + lane < p.block ? out_at(b * p.block + i * 32 + lane) : 0.f;
            top = larger(top, fabsf(y[i]));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int code = scale_code(top, p.e5m2);
        const float inv = scale_inverse(code);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * 32 + lane < p.block)
                p.codes[row * p.ld_codes + b * p.block + i * 32 + lane] = (uint8_t)codes_of(y[i] * inv, 0.f, p.e5m2);
        if (lane == 0) p.scales[row * p.ld_scales + b] = (uint8_t)code;
    }
}

// ------------------------------------------------------------------------------ gradient

struct NormBwdParams {
    const char *gy, *gh, *h, *w;  // gh, w may be NULL
    char* dx;
    int64_t ld_gy, ld_gh, ld_h, ld_dx;  // bytes
    float* dw;                    // NULL without w
    float* partial;               // [parts][cols]
    float2* stats;                // [rows] (s, s^3 mean(g h)), the general path's
    int64_t rows;
    int32_t cols, parts;
    float eps;
};

// One row per block at a time; a thread keeps its columns' sums for dw over all
// of the block's rows, and the next row's loads are in flight during this one.
template <int KIND, int W, int NV>
__global__ void __launch_bounds__(512) k_add_norm_bwd(const NormBwdParams p) {
    typedef Unit<KIND, W> U;
    constexpr int ES = sizeof(typename Num<KIND>::T), B = W * ES;
    __shared__ float s_sum[2][32][2];  // two rows' sums take turns: one barrier a row
    griddep_wait();
    const int G = blockDim.x, j = threadIdx.x, units = p.cols / W;
    U w[NV], g[NV], h[NV], gh[NV];
    float dw[NV][W];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        w[i].zero();
        if (p.w && j + i * G < units) w[i].load(p.w + (int64_t)(j + i * G) * B);
#pragma unroll
        for (int k = 0; k < W; ++k) dw[i][k] = 0.f;
    }
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t at = (int64_t)(j + i * G) * B;
            g[i].zero(), h[i].zero(), gh[i].zero();
            if (row < p.rows && j + i * G < units) {
                g[i].load(p.gy + row * p.ld_gy + at);
                h[i].load(p.h + row * p.ld_h + at);
                if (p.gh) gh[i].load(p.gh + row * p.ld_gh + at);
            }
        }
    };
    load(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        U g0[NV], h0[NV], gh0[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) g0[i] = g[i], h0[i] = h[i], gh0[i] = gh[i];
        load(row + gridDim.x);
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float a[W], b[W], c[W];
            g0[i].get(a), h0[i].get(b), w[i].get(c);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                sum[0] += b[k] * b[k];
                sum[1] += (p.w ? a[k] * c[k] : a[k]) * b[k];
            }
        }
        row_sums(sum, G, s_sum[turn]);
        const float s = 1.f / sqrtf(sum[0] / (float)p.cols + p.eps), m = sum[1] / (float)p.cols * s * s;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float a[W], b[W], c[W], d[W];
            g0[i].get(a), h0[i].get(b), w[i].get(c), gh0[i].get(d);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                dw[i][k] += a[k] * (b[k] * s);
                d[k] += s * ((p.w ? a[k] * c[k] : a[k]) - b[k] * m);
            }
            if (j + i * G < units) U::store(p.dx + row * p.ld_dx + (int64_t)(j + i * G) * B, d);
        }
    }
    if (!p.w) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (j + i * G < units)
#pragma unroll
            for (int k = 0; k < W; ++k) p.partial[(int64_t)blockIdx.x * p.cols + (j + i * G) * W + k] = dw[i][k];
}

// Any width and address: first the rows' two numbers, then dx and the sums for
// dw column by column, p.parts runs of rows side by side.
template <int KIND>
__global__ void __launch_bounds__(kAnyThreads) k_add_norm_stats(const NormBwdParams p) {
    typedef typename Num<KIND>::T T;
    __shared__ float s_sum[32][2];
    griddep_wait();
    const int64_t row = blockIdx.x;
    const T* const gy = reinterpret_cast<const T*>(p.gy + row * p.ld_gy);
    const T* const h = reinterpret_cast<const T*>(p.h + row * p.ld_h);
    const T* const w = reinterpret_cast<const T*>(p.w);
    float sum[2] = {0.f, 0.f};
#pragma unroll 4
    for (int c = threadIdx.x; c < p.cols; c += kAnyThreads) {
        const float a = Num<KIND>::get(sbt_ld(gy + c)), b = Num<KIND>::get(sbt_ld(h + c));
        sum[0] += b * b;
        sum[1] += (w ? a * Num<KIND>::get(sbt_ld(w + c)) : a) * b;
    }
    row_sums(sum, kAnyThreads, s_sum);
    if (threadIdx.x == 0) {
        const float s = 1.f / sqrtf(sum[0] / (float)p.cols + p.eps);
        p.stats[row] = make_float2(s, sum[1] / (float)p.cols * s * s);
    }
}

template <int KIND>
__global__ void __launch_bounds__(kAnyThreads) k_add_norm_bwd_any(const NormBwdParams p) {
    typedef typename Num<KIND>::T T;
    griddep_wait();
    const int64_t c = (int64_t)blockIdx.x * kAnyThreads + threadIdx.x;
    if (c >= p.cols) return;
    const float w = p.w ? Num<KIND>::get(sbt_ld(reinterpret_cast<const T*>(p.w) + c)) : 1.f;
    float dw = 0.f;
    const int64_t r0 = p.rows * blockIdx.y / p.parts, r1 = p.rows * (blockIdx.y + 1) / p.parts;
#pragma unroll 4
    for (int64_t row = r0; row < r1; ++row) {
        const float a = Num<KIND>::get(sbt_ld(reinterpret_cast<const T*>(p.gy + row * p.ld_gy) + c));
        const float b = Num<KIND>::get(sbt_ld(reinterpret_cast<const T*>(p.h + row * p.ld_h) + c));
        const float d = p.gh ? Num<KIND>::get(sbt_ld(reinterpret_cast<const T*>(p.gh + row * p.ld_gh) + c)) : 0.f;
        const float2 st = sbt_ld(p.stats + row);
        dw += a * (b * st.x);
        reinterpret_cast<T*>(p.dx + row * p.ld_dx)[c] = Num<KIND>::put(d + st.x * (a * w - b * st.y));
    }
    if (p.w) p.partial[(int64_t)blockIdx.y * p.cols + c] = dw;
}

// dw = the parts' sums: 32 warps take every 32nd part of 32 columns, then their
// sums are added in order.
__global__ void __launch_bounds__(1024) k_add_norm_dw(const NormBwdParams p) {
    __shared__ float s[32][33];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < p.cols)
#pragma unroll 4
        for (int i = warp; i < p.parts; i += 32) sum += sbt_ld(p.partial + (int64_t)i * p.cols + c);
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < p.cols) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][lane];
        p.dw[c] = t;
    }
}

// Rows of `ld` bytes that may be read and written as 16-byte vectors (or are absent).
bool vectors(const void* p, int64_t ld) { return !p || (sbt_aligned16(p) && ld % 16 == 0); }

int threads_for(int64_t units, int most) {
    int g = 32;
    while (g < most && g < units) g *= 2;
    return g;
}

template <int KIND, int W, int NV, bool SHIFT = false>
sbt_status launch_forward(sbt_context* ctx, NormParams& p, int G, cudaStream_t stream) {
    p.group = G;
    const int threads = std::max(G, 128), per = threads / G;
    const int64_t grid = G > 32 ? p.rows : sbt_cdiv(p.rows, per);
    const int block = G > 32 ? G : threads;
    cudaError_t e;
    if (W == 8 && p.codes)
        e = sbt_launch_dependent(k_add_norm<KIND, W, NV, W == 8 && !SHIFT, SHIFT>, dim3((unsigned)grid), dim3(block), 0, stream, p);
    else
        e = sbt_launch_dependent(k_add_norm<KIND, W, NV, false, SHIFT>, dim3((unsigned)grid), dim3(block), 0, stream, p);
    if (sbt_status st = sbt_cuda_check(e, "add_rms_norm launch")) return st;
    return sbt_after_launch(ctx, "add_rms_norm");
}

template <int KIND>
sbt_status forward(sbt_context* ctx, NormParams& p, cudaStream_t stream) {
    const bool vec = p.cols % 8 == 0 && vectors(p.x, p.ld_x) && vectors(p.r, p.ld_r) &&
                     vectors(p.h, p.ld_h) && vectors(p.y, p.ld_y) && sbt_aligned16(p.w) &&
                     (!p.codes || (((uintptr_t)p.codes | (uintptr_t)p.ld_codes) & 7) == 0);
    const bool few = p.rows <= 2 * ctx->sm_count;
    if (vec && p.cols <= 8 * 4 * 512) {
        const int units = p.cols / 8, G = threads_for(few ? units : sbt_cdiv(units, 4), few ? 1024 : 512);
        if (units <= G) return launch_forward<KIND, 8, 1>(ctx, p, G, stream);
        if (units <= 2 * G) return launch_forward<KIND, 8, 2>(ctx, p, G, stream);
        return launch_forward<KIND, 8, 4>(ctx, p, G, stream);
    }
    // the same phase everywhere: rows a whole number of vectors apart in all arrays, or equally far and equally placed
    constexpr int B = 8 * (KIND == kF32 ? 4 : 2);
    auto like_x = [&](const void* q, int64_t ld) {
        return !q || (((uintptr_t)q ^ (uintptr_t)p.x) % B == 0 && (ld - p.ld_x) % B == 0);
    };
    if (!p.codes && p.cols >= 64 && p.cols <= 8 * 2 * 1024 - 16 && like_x(p.r, p.ld_r) && like_x(p.h, p.ld_h) && like_x(p.y, p.ld_y)) {
        const int units = p.cols / 8 + 2, G = threads_for(few ? units : sbt_cdiv(units, 2), 1024);
        if (units <= G) return launch_forward<KIND, 8, 1, true>(ctx, p, G, stream);
        return launch_forward<KIND, 8, 2, true>(ctx, p, G, stream);
    }
    if (!p.codes && p.cols <= 16 * 1024) {
        const int G = threads_for(sbt_cdiv(p.cols, few ? 4 : 16), 1024);
        if (p.cols <= 4 * G) return launch_forward<KIND, 1, 4>(ctx, p, G, stream);
        return launch_forward<KIND, 1, 16>(ctx, p, G, stream);
    }
    if (sbt_status st = sbt_cuda_check(sbt_launch_dependent(k_add_norm_any<KIND>, dim3((unsigned)p.rows),
                                                            dim3(kAnyThreads), 0, stream, p),
                                       "add_rms_norm launch"))
        return st;
    return sbt_after_launch(ctx, "add_rms_norm");
}

// The gradient's forms: rows in registers as vectors or element by element (threads a row), or the general one.
constexpr int kVectorCols = 8 * 2 * 512, kElementCols = 8 * 512;
int vector_threads(int32_t cols) { return threads_for(sbt_cdiv(cols / 8, 2), 512); }
int element_threads(int32_t cols) { return threads_for(sbt_cdiv(cols, 8), 512); }
// Rows of partial sums for dw.  512 threads an SM: the registers of two rows' loads and of the sums for dw.
int register_parts(const sbt_context* ctx, int64_t rows, int G) {
    return (int)std::min<int64_t>(rows, std::max<int64_t>(1, (int64_t)ctx->sm_count * std::max(1, 512 / G)));
}
int general_parts(const sbt_context* ctx, int64_t rows, int32_t cols) {
    return (int)std::min<int64_t>(rows, std::max<int64_t>(1, 4 * ctx->sm_count / sbt_cdiv(cols, kAnyThreads)));
}
// The most that a call of these extents writes: addresses and strides say which form it takes.
int most_parts(const sbt_context* ctx, int64_t rows, int32_t cols) {
    int n = 0;
    if (cols % 8 == 0 && cols <= kVectorCols) n = register_parts(ctx, rows, vector_threads(cols));
    return std::max(n, cols <= kElementCols ? register_parts(ctx, rows, element_threads(cols)) : general_parts(ctx, rows, cols));
}

template <int KIND, int W, int NV>
sbt_status launch_backward(sbt_context* ctx, NormBwdParams& p, int G, cudaStream_t stream) {
    p.parts = register_parts(ctx, p.rows, G);
    if (sbt_status st = sbt_cuda_check(sbt_launch_dependent(k_add_norm_bwd<KIND, W, NV>, dim3(p.parts), dim3(G), 0,
                                                            stream, p),
                                       "add_rms_norm_backward launch"))
        return st;
    return sbt_after_launch(ctx, "add_rms_norm_backward");
}

template <int KIND>
sbt_status backward(sbt_context* ctx, NormBwdParams& p, cudaStream_t stream) {
    const bool vec = p.cols % 8 == 0 && vectors(p.gy, p.ld_gy) && vectors(p.gh, p.ld_gh) &&
                     vectors(p.h, p.ld_h) && vectors(p.dx, p.ld_dx) && sbt_aligned16(p.w);
    sbt_status st = SBT_OK;
    if (p.rows == 0) {
        p.parts = 0;
    } else if (vec && p.cols <= kVectorCols) {
        const int units = p.cols / 8, G = vector_threads(p.cols);
        st = units <= G ? launch_backward<KIND, 8, 1>(ctx, p, G, stream) : launch_backward<KIND, 8, 2>(ctx, p, G, stream);
    } else if (p.cols <= kElementCols) {
        const int G = element_threads(p.cols);
        st = p.cols <= 4 * G ? launch_backward<KIND, 1, 4>(ctx, p, G, stream)
                             : launch_backward<KIND, 1, 8>(ctx, p, G, stream);
    } else {
        if ((st = sbt_cuda_check(sbt_launch_dependent(k_add_norm_stats<KIND>, dim3((unsigned)p.rows),
                                                      dim3(kAnyThreads), 0, stream, p),
                                 "add_rms_norm_backward launch")) ||
            (st = sbt_after_launch(ctx, "add_rms_norm_backward")))
            return st;
        const int64_t blocks = sbt_cdiv(p.cols, kAnyThreads);
        p.parts = general_parts(ctx, p.rows, p.cols);
        if ((st = sbt_cuda_check(sbt_launch_dependent(k_add_norm_bwd_any<KIND>, dim3((unsigned)blocks, p.parts),
                                                      dim3(kAnyThreads), 0, stream, p),
                                 "add_rms_norm_backward launch")) == SBT_OK)
            st = sbt_after_launch(ctx, "add_rms_norm_backward");
    }
    if (st || !p.w) return st;
    if ((st = sbt_cuda_check(sbt_launch_dependent(k_add_norm_dw, dim3((unsigned)sbt_cdiv(p.cols, 32)), dim3(1024), 0,
                                                  stream, p),
                             "add_rms_norm_backward dweight launch")))
        return st;
    return sbt_after_launch(ctx, "add_rms_norm_backward dweight");
}

}  // namespace

sbt_status sbt_launch_add_norm(sbt_context* ctx, sbt_dtype dtype, const SbtRows& x, const SbtRows& r, int64_t rows,
                               int32_t cols, const void* w, float eps, const SbtRows& h, const SbtRows& y,
                               const sbt_code_rows* codes, cudaStream_t stream) {
    const int es = sbt_dtype_size(dtype);
    NormParams p = {};
    p.x = (const char*)x.p, p.ld_x = x.ld * es;
    p.r = (const char*)r.p, p.ld_r = r.ld * es;
    p.h = (char*)const_cast<void*>(h.p), p.ld_h = h.ld * es;
    p.y = (char*)const_cast<void*>(y.p), p.ld_y = y.ld * es;
    p.w = (const char*)w;
    p.rows = rows, p.cols = cols, p.eps = eps;
    if (codes) {
        p.codes = (uint8_t*)codes->codes, p.scales = codes->scales;
        p.ld_codes = codes->ld, p.ld_scales = codes->ld_scale;
        p.block = codes->block, p.e5m2 = codes->format == SBT_FMT_E5M2;
    }
    switch (kind_of(dtype)) {
        case kF32: return forward<kF32>(ctx, p, stream);
        case kBF16: return forward<kBF16>(ctx, p, stream);
        default: return forward<kF16>(ctx, p, stream);
    }
}

// The parts of dw, then the general form's numbers per row, which rows that fit registers without vectors never need.
static size_t parts_bytes(const sbt_context* ctx, int64_t rows, int32_t cols) {
    return (size_t)sbt_cdiv((int64_t)most_parts(ctx, rows, cols) * cols * 4, 256) * 256;
}
size_t sbt_add_norm_bwd_bytes(const sbt_context* ctx, int64_t rows, int32_t cols) {
    return parts_bytes(ctx, rows, cols) + (cols > kElementCols ? (size_t)rows * sizeof(float2) : 0);
}

sbt_status sbt_launch_add_norm_bwd(sbt_context* ctx, sbt_dtype dtype, const SbtRows& gy, const SbtRows& gh,
                                   const SbtRows& h, int64_t rows, int32_t cols, const void* w, float eps,
                                   const SbtRows& dx, float* dw, void* workspace, cudaStream_t stream) {
    const int es = sbt_dtype_size(dtype);
    NormBwdParams p = {};
    p.gy = (const char*)gy.p, p.ld_gy = gy.ld * es;
    p.gh = (const char*)gh.p, p.ld_gh = gh.ld * es;
    p.h = (const char*)h.p, p.ld_h = h.ld * es;
    p.dx = (char*)const_cast<void*>(dx.p), p.ld_dx = dx.ld * es;
    p.w = (const char*)w, p.dw = dw;
    p.rows = rows, p.cols = cols, p.eps = eps;
    p.partial = (float*)workspace;
    p.stats = (float2*)((char*)workspace + parts_bytes(ctx, rows, cols));
    switch (kind_of(dtype)) {
        case kF32: return backward<kF32>(ctx, p, stream);
        case kBF16: return backward<kBF16>(ctx, p, stream);
        default: return backward<kF16>(ctx, p, stream);
    }
}
