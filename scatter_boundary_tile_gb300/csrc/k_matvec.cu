// A few rows times a matrix of 4-bit weights with group scales:
//   y[t][n] = alpha sum_k x[t][k] w[k][n] s[k / group][n],
// w in E2M1, two columns a byte, s in E8M0 or E4M3.
//
// The weights are read once and bound the call: 0.5 byte each, so at the copy
// rate an SM has to turn ~47 of them a clock into numbers and multiply them for
// up to 16 rows.  The products run on mma.sync m16n8k16 (fp16 in, fp32 sums):
// 16 columns of w by 8 rows of x, 16 k.  E2M1 is exact in fp16 and has a
// conversion of two codes at once; a tcgen05 tile would want the weights as
// fp16 in shared memory, written there by the same instructions and read again.
//
// A column's neighbour lies in the same byte, but the conversion and the matrix
// instruction want pairs along k: two bytes of rows k and k + 1 trade nibbles
// (4 operations for 16 weights), the even column's pair to row g of the tile
// and the odd column's to row g + 8.  The k of a step are numbered so that a
// lane's four are neighbours, for the weights and for x alike.
//
// Groups.  The products of U k (32, or 16) are summed by the matrix unit and
// added to the running sums times the group's scale.
//
// x.  fp16 enters as it is.  bf16 and fp32 are scaled by a power of two to
// below 2^15, per row and for the k seen so far (as the running maximum of a
// softmax: when it grows, the sums are scaled), and enter as one and two fp16
// numbers; bf16's 8 bits fit in fp16's 11 unless they are below its last step,
// 2^-39 of the largest.
//
// Split.  A block has 256 columns and a share of k, its warps a share each;
// every warp has a private ring of stages filled by cp.async and waits for no
// other until the end.  A cluster of up to eight blocks shares the k of one
// tile; warps, then blocks, join in a fixed order through shared memory.
#include <algorithm>

#include "sbt_internal.cuh"
#include "sbt_num.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace sbt_num;
using sbt_ptx::griddep_wait;

constexpr int kWarps = 8, kCols = 256, kClusterMost = 8;
constexpr int kPitch = kCols + 20;  // floats between rows of partial sums: lanes of a half warp meet no bank twice
constexpr int kFixedStages = 4;     // what a block costs besides its stages, in stages

struct MatvecParams {
    const char* x;
    const uint8_t *w, *s;
    char* y;
    int64_t ld_x, ld_w, ld_s, ld_y;  // bytes
    int64_t tokens, N, K, group;
    float alpha;
    int32_t y_kind, ranks, x_vec;
};

template <int KIND, int U, bool ALIGNED>
struct Shape {
    static constexpr int ES = sizeof(typename Num<KIND>::T);
    static constexpr int PITCH = ALIGNED ? 128 : 144;      // bytes of a row of weights in a stage
    static constexpr int STAGE = U * PITCH + 288;          // and up to 256 + 15 bytes of scales
    static constexpr int STAGES = (112 << 10) / (kWarps * STAGE);
    static constexpr int RING = STAGES * STAGE;
    static constexpr size_t SMEM = (size_t)kWarps * (RING > 8 * kPitch * 4 ? RING : 8 * kPitch * 4);
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four bytes of two E2M1 codes each as fp16 pairs.
__device__ __forceinline__ void unpack_e2m1(uint32_t v, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(v));
}

// Two scales.
template <bool E4M3>
__device__ __forceinline__ float2 unpack_scales(uint32_t two) {
    uint32_t h;
    if (E4M3) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
        return __half22float2(*reinterpret_cast<const __half2*>(&h));
    }
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// KIND: of x.  U: k of a stage.  MT: 8 rows of x each.
template <int KIND, int U, bool E4M3, int MT, bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps, MT == 1 ? 2 : 1) k_matvec(const MatvecParams p) {
    typedef Shape<KIND, U, ALIGNED> S;
    typedef typename Num<KIND>::T T;
    constexpr int STEPS = U / 16, TERMS = KIND == kF32 ? 2 : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % p.ranks;
    const int64_t tile = blockIdx.x / p.ranks, n0 = tile * kCols, tok0 = (int64_t)blockIdx.y * 8 * MT;
    const int64_t units = p.K / U, workers = (int64_t)kWarps * p.ranks, me = (int64_t)rank * kWarps + warp;
    const int64_t u0 = units * me / workers, u1 = units * (me + 1) / workers;
    uint8_t* const ring = smem + warp * S::RING;
    const uint32_t ring_u32 = sbt_ptx::smem_u32(ring);
    griddep_wait();

    // ---- copies: rows of 128 bytes of weights, and the group's 256 scales, nothing past their ends
    const int w_bytes = (int)min((int64_t)(kCols / 2), (p.N + 1) / 2 - n0 / 2), s_bytes = (int)min((int64_t)kCols, p.N - n0);
    auto copy = [&](int64_t u, int stage) {
        const uint32_t dst = ring_u32 + stage * S::STAGE;
        const uint8_t* const src = p.w + u * U * p.ld_w + n0 / 2;
        if (ALIGNED) {
            const int c = lane & 7, bytes = min(max(w_bytes - c * 16, 0), 16);
#pragma unroll
            for (int i = 0; i < U / 4; ++i) {
                const int r = i * 4 + (lane >> 3);
                copy16(dst + r * 128 + ((c ^ (((r >> 2) & 3) << 1)) << 4), bytes ? src + r * p.ld_w + c * 16 : p.w, bytes);
            }
        } else {
            const int c = lane & 15;  // nine pieces cover a row from the 16-byte boundary before it
#pragma unroll 4
            for (int i = 0; i < U / 2; ++i) {
                const int r = i * 2 + (lane >> 4);
                const uint8_t* const a = src + r * p.ld_w;
                const int shift = (int)((uintptr_t)a & 15), bytes = min(max(shift + w_bytes - c * 16, 0), 16);
                if (bytes) copy16(dst + r * 144 + c * 16, a - shift + c * 16, bytes);
            }
        }
        const uint8_t* const a = p.s + u * U / p.group * p.ld_s + n0;
        const int shift = (int)((uintptr_t)a & 15), bytes = min(max(shift + s_bytes - lane * 16, 0), 16);
        if (bytes) copy16(dst + U * S::PITCH + lane * 16, a - shift + lane * 16, bytes);
    };

    // ---- x: this lane's four k of each step, of rows tok0 + 8 m + g; the next stage's while this one is used
    struct Raw {
        T v[4];
    };
    auto load_x = [&](int64_t u, Raw (&r)[STEPS][MT]) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int64_t tok = tok0 + m * 8 + g;
                const T* const a = reinterpret_cast<const T*>(p.x + tok * p.ld_x) + u * U + s * 16 + t * 4;
                if (u >= u1 || tok >= p.tokens) {
                    r[s][m] = Raw{};
                } else if (p.x_vec) {
                    if constexpr (KIND == kF32)
                        *reinterpret_cast<uint4*>(&r[s][m]) = sbt_ld(reinterpret_cast<const uint4*>(a));
                    else
                        *reinterpret_cast<uint2*>(&r[s][m]) = sbt_ld(reinterpret_cast<const uint2*>(a));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[s][m].v[i] = sbt_ld(a + i);
                }
            }
    };

    float sum[MT][16][4];  // columns g*32 + 2 i, + 1; rows 2 t, + 1 of x
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[m][i][k] = 0.f;
    int exponent[MT];  // x of row g enters as x 2^-exponent
#pragma unroll
    for (int m = 0; m < MT; ++m) exponent[m] = -126;

    Raw raw[STEPS][MT];
    load_x(u0, raw);
#pragma unroll 1
    for (int i = 0; i < S::STAGES - 1; ++i) {
        if (u0 + i < u1) copy(u0 + i, i);
        copy_commit();
    }
    int stage = 0;
#pragma unroll 1
    for (int64_t u = u0; u < u1; ++u) {
        copy_wait<S::STAGES - 2>();
        __syncwarp();
        if (u + S::STAGES - 1 < u1) copy(u + S::STAGES - 1, stage == 0 ? S::STAGES - 1 : stage - 1);
        copy_commit();

        // x as fp16 pairs along k
        uint32_t b[STEPS][MT][TERMS][2];
        if constexpr (KIND == kF16) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint2 v = *reinterpret_cast<const uint2*>(&raw[s][m]);
                    b[s][m][0][0] = v.x, b[s][m][0][1] = v.y;
                }
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                // exponent of the largest finite |x| of the row in this stage
                int top = 0;
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = (int)(__float_as_uint(Num<KIND>::get(raw[s][m].v[i])) >> 23) & 255;
                        top = max(top, e == 255 ? 0 : e);
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int want = max(top - 127 - 14, -126);
                if (__any_sync(0xffffffffu, want > exponent[m])) {
                    const int now = max(want, exponent[m]), gap = min(now - exponent[m], 127);
                    exponent[m] = now;
                    // the rows of the sums are 2 t and 2 t + 1, held by lanes 8 t and 8 t + 4
                    const float f0 = power(-__shfl_sync(0xffffffffu, gap, 8 * t));
                    const float f1 = power(-__shfl_sync(0xffffffffu, gap, 8 * t + 4));
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        sum[m][i][0] *= f0, sum[m][i][1] *= f1;
                        sum[m][i][2] *= f0, sum[m][i][3] *= f1;
                    }
                }
                const float f = power(-exponent[m]);
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float lo = Num<KIND>::get(raw[s][m].v[2 * i]) * f, hi = Num<KIND>::get(raw[s][m].v[2 * i + 1]) * f;
                        const __half2 h = __floats2half2_rn(lo, hi);
                        b[s][m][0][i] = *reinterpret_cast<const uint32_t*>(&h);
                        if constexpr (TERMS == 2) {
                            const float2 q = __half22float2(h);
                            // what the first number leaves; nothing of an infinity
                            const __half2 r = __floats2half2_rn(isinf(lo) ? 0.f : lo - q.x, isinf(hi) ? 0.f : hi - q.y);
                            b[s][m][TERMS - 1][i] = *reinterpret_cast<const uint32_t*>(&r);
                        }
                    }
            }
        }
        load_x(u + 1, raw);

        // weights: rows 16 s + 4 t + r, columns g*32 .. + 31
        uint32_t w[STEPS][4][4];
        const uint8_t* const st = ring + stage * S::STAGE;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * s + 4 * t + r;
                if (ALIGNED) {
                    const uint4 v = *reinterpret_cast<const uint4*>(st + row * 128 + ((g ^ (((row >> 2) & 3) << 1)) << 4));
                    w[s][r][0] = v.x, w[s][r][1] = v.y, w[s][r][2] = v.z, w[s][r][3] = v.w;
                } else {
                    const int shift = (int)((uintptr_t)(p.w + (u * U + row) * p.ld_w + n0 / 2) & 15);
                    const uint32_t* const q = reinterpret_cast<const uint32_t*>(st + row * 144 + g * 16 + (shift & ~3));
                    uint32_t a = q[0];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t c = q[j + 1];
                        w[s][r][j] = __funnelshift_r(a, c, (shift & 3) * 8);
                        a = c;
                    }
                }
            }
        uint32_t sc[8];
        {
            const int shift = (int)((uintptr_t)(p.s + u * U / p.group * p.ld_s + n0) & 15);
            const uint8_t* const a = st + U * S::PITCH + g * 32;
            if (shift == 0) {
                const uint4 v0 = *reinterpret_cast<const uint4*>(a), v1 = *reinterpret_cast<const uint4*>(a + 16);
                sc[0] = v0.x, sc[1] = v0.y, sc[2] = v0.z, sc[3] = v0.w;
                sc[4] = v1.x, sc[5] = v1.y, sc[6] = v1.z, sc[7] = v1.w;
            } else {
                const uint32_t* const q = reinterpret_cast<const uint32_t*>(a + (shift & ~3));
                uint32_t c = q[0];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t d = q[j + 1];
                    sc[j] = __funnelshift_r(c, d, (shift & 3) * 8);
                    c = d;
                }
            }
        }
        // a byte of the last words may be past the scales and the weights: columns past N, which nobody reads
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a[STEPS][4][4];  // [step][fragment][column pair]
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t lo = w[s][2 * k][j], hi = w[s][2 * k + 1][j];
                    unpack_e2m1((lo & 0x0F0F0F0Fu) | ((hi << 4) & 0xF0F0F0F0u), a[s][2 * k]);
                    unpack_e2m1(((lo >> 4) & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u), a[s][2 * k + 1]);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack_scales<E4M3>(i & 1 ? sc[2 * j + i / 2] >> 16 : sc[2 * j + i / 2]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
                        const uint32_t frag[4] = {a[s][0][i], a[s][1][i], a[s][2][i], a[s][3][i]};
#pragma unroll
                        for (int q = 0; q < TERMS; ++q) mma(c, frag, b[s][m][q][0], b[s][m][q][1]);
                    }
                    float(&d)[4] = sum[m][4 * j + i];
                    d[0] = fmaf(c[0], f.x, d[0]), d[1] = fmaf(c[1], f.x, d[1]);
                    d[2] = fmaf(c[2], f.y, d[2]), d[3] = fmaf(c[3], f.y, d[3]);
                }
            }
        }
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
    }
    copy_wait<0>();

    // ---- the warps' sums, then the blocks': a block finishes every p.ranks-th row
    float* const part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        float f0 = 1.f, f1 = 1.f;
        if (KIND != kF16) {
            f0 = power(__shfl_sync(0xffffffffu, exponent[m], 8 * t));
            f1 = power(__shfl_sync(0xffffffffu, exponent[m], 8 * t + 4));
        }
        __syncthreads();
        float* const mine = part + warp * 8 * kPitch;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = g * 34 + 2 * i;
            const float(&d)[4] = sum[m][i];
            *reinterpret_cast<float2*>(mine + (2 * t) * kPitch + n) = make_float2(d[0] * f0, d[2] * f0);
            *reinterpret_cast<float2*>(mine + (2 * t + 1) * kPitch + n) = make_float2(d[1] * f1, d[3] * f1);
        }
        __syncthreads();
        const int n = threadIdx.x, at = (n >> 5) * 34 + (n & 31);
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            v[r] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v[r] += part[(w * 8 + r) * kPitch + at];
        }
        if (p.ranks > 1) {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 8; ++r) part[r * kPitch + at] = v[r];
            sbt_ptx::cluster_sync();
        }
        auto put = [&](int r, float x) {
            const int64_t tok = tok0 + m * 8 + r;
            if (tok >= p.tokens || n0 + n >= p.N) return;
            char* const y = p.y + tok * p.ld_y;
            x *= p.alpha;
            if (p.y_kind == kF32)
                reinterpret_cast<float*>(y)[n0 + n] = x;
            else
                reinterpret_cast<uint16_t*>(y)[n0 + n] = p.y_kind == kBF16 ? Num<kBF16>::put(x) : Num<kF16>::put(x);
        };
        if (p.ranks == 1) {
#pragma unroll
            for (int r = 0; r < 8; ++r) put(r, v[r]);
        } else {
            const uint32_t from = sbt_ptx::smem_u32(part + at);
            for (int r = rank; r < 8 && tok0 + m * 8 + r < p.tokens; r += p.ranks) {
                float x = 0.f;
                for (int q = 0; q < p.ranks; ++q) {
                    float part_q;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(part_q)
                                 : "r"(sbt_ptx::mapa_shared(from + r * kPitch * 4, q)));
                    x += part_q;
                }
                put(r, x);
            }
            __syncwarp();
            sbt_ptx::cluster_sync();  // nobody leaves, or writes the next rows' sums, while another reads
        }
    }
}

template <int KIND, int U, bool E4M3, int MT, bool ALIGNED>
sbt_status launch(sbt_context* ctx, MatvecParams& p, cudaStream_t stream) {
    constexpr auto kern = k_matvec<KIND, U, E4M3, MT, ALIGNED>;
    constexpr size_t smem = Shape<KIND, U, ALIGNED>::SMEM;
    const int slots = sbt_resident_blocks<kern>(ctx, 32 * kWarps, smem);
    const int64_t tiles = sbt_cdiv(p.N, kCols), chunks = sbt_cdiv(p.tokens, 8 * MT), units = p.K / U;
    // Blocks per tile: the number with which the last wave's end comes first.
    int64_t best = INT64_MAX;
    for (int c = 1; c <= kClusterMost && (c == 1 || c * kWarps <= units); ++c) {
        const int64_t cost = sbt_cdiv(tiles * chunks * c, slots) * (sbt_cdiv(units, (int64_t)c * kWarps) + kFixedStages);
        if (cost < best) best = cost, p.ranks = c;
    }
    if (sbt_status st = sbt_cuda_check(
            sbt_launch_dependent_cluster(kern, dim3((unsigned)(tiles * p.ranks), (unsigned)chunks), dim3(32 * kWarps),
                                         (unsigned)p.ranks, smem, stream, p),
            "matvec_e2m1 launch"))
        return st;
    return sbt_after_launch(ctx, "matvec_e2m1");
}

template <int KIND, int U, bool E4M3, int MT>
sbt_status pick_aligned(sbt_context* ctx, MatvecParams& p, cudaStream_t stream) {
    return sbt_aligned16(p.w) && p.ld_w % 16 == 0 ? launch<KIND, U, E4M3, MT, true>(ctx, p, stream)
                                                  : launch<KIND, U, E4M3, MT, false>(ctx, p, stream);
}

template <int KIND>
sbt_status pick(sbt_context* ctx, MatvecParams& p, bool e4m3, cudaStream_t stream) {
    p.x_vec = ((uintptr_t)p.x | (uintptr_t)p.ld_x) % (KIND == kF32 ? 16 : 8) == 0;
    const bool wide = p.group % 32 == 0, two = p.tokens > 8;
    if (wide && e4m3) return two ? pick_aligned<KIND, 32, true, 2>(ctx, p, stream) : pick_aligned<KIND, 32, true, 1>(ctx, p, stream);
    if (wide) return two ? pick_aligned<KIND, 32, false, 2>(ctx, p, stream) : pick_aligned<KIND, 32, false, 1>(ctx, p, stream);
    if (e4m3) return two ? pick_aligned<KIND, 16, true, 2>(ctx, p, stream) : pick_aligned<KIND, 16, true, 1>(ctx, p, stream);
    return two ? pick_aligned<KIND, 16, false, 2>(ctx, p, stream) : pick_aligned<KIND, 16, false, 1>(ctx, p, stream);
}

}  // namespace

sbt_status sbt_launch_matvec(sbt_context* ctx, sbt_dtype dtype, const SbtRows& x, int64_t tokens, const void* B,
                             int64_t ldb, bool e4m3_scales, const void* scales, int64_t ld_sb, int64_t K_s,
                             float alpha, const SbtRows& y, sbt_dtype y_dtype, int64_t N, int64_t K,
                             cudaStream_t stream) {
    MatvecParams p = {};
    p.x = (const char*)x.p, p.ld_x = x.ld * sbt_dtype_size(dtype);
    p.w = (const uint8_t*)B, p.ld_w = ldb / 2;
    p.s = (const uint8_t*)scales, p.ld_s = ld_sb;
    p.y = (char*)const_cast<void*>(y.p), p.ld_y = y.ld * sbt_dtype_size(y_dtype);
    p.tokens = tokens, p.N = N, p.K = K, p.group = K ? K / K_s : 32;
    p.alpha = alpha, p.y_kind = kind_of(y_dtype);
    switch (kind_of(dtype)) {
        case kF32: return pick<kF32>(ctx, p, e4m3_scales, stream);
        case kBF16: return pick<kBF16>(ctx, p, e4m3_scales, stream);
        default: return pick<kF16>(ctx, p, e4m3_scales, stream);
    }
}
