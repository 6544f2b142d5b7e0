// Paged attention, 16-bit caches: the tile math on the tensor cores.
//
// S^T = K Q^T and O^T += V^T P^T: positions (then head elements) are the
// 16-row side of mma.m16n8k16 and the query heads of one key-value head its
// 8-column side, so one to eight heads cost one column block.  The operation
// reads every key and value once and does 2 x 8 multiply-adds with each, 54
// TFLOP/s at the copy peak for one column block: memory bounds it, the mma.sync rate is
// far above what it asks, and operands of 16 rows a warp let every warp run
// its own softmax without waiting for a 128-row tile.
//
// The second product takes 16-bit operands, and one rounding of a probability
// to 2^-8 (bf16) or 2^-11 (fp16) would cost as much as the output's own.  So a
// probability is split in two 16-bit numbers, p = hi + lo to 2^-16 or 2^-22,
// and multiplied twice.  fp16 has few exponents: p = 2^(s - m) <= 1 would be
// subnormal below 2^-14 and nothing below 2^-25, while l, summed from the fp32
// values, still counts it.  There p enters as 2^15 p <= 32768, and o is brought
// back by 2^-15 (exact) where it leaves the registers: steps of 2^-39.  Against
// one rounded product of p itself the fp16 output's error falls from 1.19 to 1.00
// of one rounding; 128 sequences to 8192 with 128 / 8 heads 352.9 -> 355.7 us, head
// size 256 with 16 heads per key 217.7 -> 226.6, others within 1.5 % (4 % at 32 per key).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "k_paged_attention.cuh"

namespace {

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool BF>
__device__ __forceinline__ void mma16(float* c, const uint32_t* a, const uint32_t* b) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <bool BF, int DP_, int NB, int MT>
struct Mma16 {
    typedef uint16_t T;
    static constexpr int ES = 2, TOK = 16 * MT, DP = DP_, HEADS = 8 * NB, SCRATCH = 0;
    static constexpr int PITCH = DP * 2;
    // the eight rows of one 8 x 8 matrix lie in different banks: rows of 128 n bytes differ in the
    // XOR of all three chunk bits, rows of 192 in their start's and two
    static constexpr bool WIDE = PITCH % 128 == 0;
    static constexpr float P_UP = BF ? 1.f : 32768.f, P_DOWN = 1.f / P_UP;  // of the probabilities in o
    static __device__ __forceinline__ int swizzle(int t) { return WIDE ? t & 7 : (t >> 1) & 3; }
    // byte of chunk 2 k + x (x = 0, 1) in a row, where s = x ^ swizzle(row)
    static __device__ __forceinline__ uint32_t chunk_at(int k, uint32_t s) {
        return WIDE ? (k >> 2) * 128 + ((s ^ (2 * (k & 3))) << 4) : (k >> 1) * 64 + ((s ^ (2 * (k & 1))) << 4);
    }
    static __device__ __forceinline__ uint16_t from_float(float x) {
        return BF ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
    }
    // two values rounded to 16 bits, the first in the low half
    static __device__ __forceinline__ uint32_t pack2(float x, float y) {
        if (BF) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            return *reinterpret_cast<const uint32_t*>(&h);
        }
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack2(uint32_t w) {
        if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }

    uint32_t qf[DP / 16][NB][2];
    float o[DP / 16][NB][4];
    float mx[NB][2], l[NB][2];

    __device__ __forceinline__ void load_q(const AttnParams& p, const AttnRow& r, int32_t row, float*) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q2 = (lane & 3) * 2;
        const int32_t kvh = row / p.n_chunks, h0 = (row - kvh * p.n_chunks) * p.chunk;
        const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
        const uint16_t* base = reinterpret_cast<const uint16_t*>(p.q) + r.b * p.ld_q + (kvh * p.group + h0) * p.ld_qh;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int h = n * 8 + g;
            const uint16_t* x = base + h * p.ld_qh;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int d = k * 16 + i * 8 + q2;
                    uint32_t w = 0;
                    if (h < heads && d < p.head_dim) {
                        if (p.q_words) {
                            w = sbt_ld(reinterpret_cast<const uint32_t*>(x + d));
                        } else {
                            w = sbt_ld(x + d);
                            if (d + 1 < p.head_dim) w |= (uint32_t)sbt_ld(x + d + 1) << 16;
                        }
                    }
                    qf[k][n][i] = w;
                }
            mx[n][0] = mx[n][1] = -CUDART_INF_F;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][n][i] = 0.f;
        }
    }

    __device__ __forceinline__ void tile(const AttnParams& p, const uint8_t*, uint32_t k_s, uint32_t v_s, uint32_t bits,
                                         float*) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        float s[MT][NB][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n) s[m][n][0] = s[m][n][1] = s[m][n][2] = s[m][n][3] = 0.f;
        const uint32_t k_row = k_s + (lane & 15) * PITCH;
        const uint32_t k_x = (lane >> 4) ^ swizzle(lane & 15);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t a[4];
                ldsm4(a, k_row + m * 16 * PITCH + chunk_at(k, k_x));
#pragma unroll
                for (int n = 0; n < NB; ++n) mma16<BF>(s[m][n], a, qf[k][n]);
            }
        constexpr uint32_t ALL = MT == 2 ? 0xffffffffu : 0xffffu;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[m][n][i] *= p.scale_log2;
        if (bits != ALL) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!((bits >> (m * 16 + g + (i >> 1) * 8)) & 1u)) s[m][n][i] = -CUDART_INF_F;
        }
        uint32_t hi[MT][NB][2], lo[MT][NB][2];
        float alpha[NB][2];
        bool grown = false;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float t = fmaxf(s[0][n][j], s[0][n][j + 2]);
#pragma unroll
                for (int m = 1; m < MT; ++m) t = fmaxf(t, fmaxf(s[m][n][j], s[m][n][j + 2]));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                t = fmaxf(t, mx[n][j]);
                const float ts = t == -CUDART_INF_F ? 0.f : t;
                alpha[n][j] = sbt_attn::exp2_fast(mx[n][j] - ts);
                grown |= t != mx[n][j];
                mx[n][j] = t;
                l[n][j] *= alpha[n][j];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    s[m][n][j] = sbt_attn::exp2_fast(s[m][n][j] - ts);
                    s[m][n][j + 2] = sbt_attn::exp2_fast(s[m][n][j + 2] - ts);
                    l[n][j] += s[m][n][j] + s[m][n][j + 2];
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float p0 = s[m][n][2 * i] * P_UP, p1 = s[m][n][2 * i + 1] * P_UP;
                    const uint32_t h = pack2(p0, p1);
                    const float2 f = unpack2(h);
                    hi[m][n][i] = transpose8(h);
                    lo[m][n][i] = transpose8(pack2(p0 - f.x, p1 - f.y));
                }
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[k][n][i] *= alpha[n][i & 1];
        }
        const int v_t = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t v_row = v_s + v_t * PITCH, v_x = ((lane >> 3) & 1) ^ swizzle(v_t);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t a[4];
                ldsm4_t(a, v_row + m * 16 * PITCH + chunk_at(k, v_x));
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    mma16<BF>(o[k][n], a, hi[m][n]);
                    mma16<BF>(o[k][n], a, lo[m][n]);
                }
            }
    }

    // l over the lanes that hold different positions of the same heads
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 4);
                l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 8);
                l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 16);
            }
    }

    // Lane (g, q) holds elements 16 k + g and 16 k + g + 8 of heads 2 q, 2 q + 1; transposed in
    // 16 bits it holds element pairs 16 k + 2 q and 16 k + 8 + 2 q of head g: four lanes write 16 bytes.
    __device__ __forceinline__ void put_row(const AttnParams& p, int32_t b, int32_t qh, int32_t heads) {
        finish();
        const int lane = threadIdx.x & 31, g = lane >> 2, q2 = (lane & 3) * 2;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (n * 8 >= heads) break;
            const float inv0 = sbt_attn::inverse(l[n][0]) * P_DOWN, inv1 = sbt_attn::inverse(l[n][1]) * P_DOWN;
            const int h = n * 8 + g;
            uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + b * p.ld_out + (int64_t)(qh + h) * p.ld_oh;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w = transpose8(pack2(o[k][n][2 * i] * inv0, o[k][n][2 * i + 1] * inv1));
                    const int d = k * 16 + i * 8 + q2;
                    if (h >= heads || d >= p.head_dim) continue;
                    if (p.out_words) {
                        *reinterpret_cast<uint32_t*>(dst + d) = w;
                    } else {
                        dst[d] = (uint16_t)w;
                        if (d + 1 < p.head_dim) dst[d + 1] = (uint16_t)(w >> 16);
                    }
                }
            if (p.lse && g == 0)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (n * 8 + q2 + j < heads)
                        p.lse[(int64_t)b * p.q_heads + qh + n * 8 + q2 + j] = sbt_attn::log_sum(mx[n][j], l[n][j]);
        }
    }

    // the state to dst [DP][HEADS] and ml [HEADS]
    __device__ __forceinline__ void put_part(float* dst, float2* ml) {
        finish();
        const int lane = threadIdx.x & 31, g = lane >> 2, q2 = (lane & 3) * 2;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float2*>(dst + (k * 16 + i * 8 + g) * HEADS + n * 8 + q2) =
                        make_float2(o[k][n][2 * i] * P_DOWN, o[k][n][2 * i + 1] * P_DOWN);
            if (g == 0)
#pragma unroll
                for (int j = 0; j < 2; ++j) ml[n * 8 + q2 + j] = make_float2(mx[n][j], l[n][j]);
        }
    }
};

template <bool BF, int DP, int MT, int STAGES, int WARPS, int BLOCKS>
sbt_status by_heads(sbt_context* ctx, const AttnParams& p, cudaStream_t stream) {
    if (p.chunk <= 8) return sbt_attention_enqueue<Mma16<BF, DP, 1, MT>, STAGES, WARPS, BLOCKS>(ctx, p, stream);
    return sbt_attention_enqueue<Mma16<BF, DP, 2, MT>, STAGES, WARPS, BLOCKS>(ctx, p, stream);
}

// Warps per block and blocks per SM: as many as two stages each leave room for.
template <bool BF>
sbt_status by_dim(sbt_context* ctx, const AttnParams& p, cudaStream_t stream) {
    if (p.head_dim <= 64) return by_heads<BF, 64, 2, 2, 4, 3>(ctx, p, stream);
    if (p.head_dim <= 96) return by_heads<BF, 96, 1, 3, 4, 3>(ctx, p, stream);
    if (p.head_dim <= 128) return by_heads<BF, 128, 1, 2, 4, 3>(ctx, p, stream);
    if (p.head_dim <= 192) return by_heads<BF, 192, 1, 2, 4, 2>(ctx, p, stream);
    return by_heads<BF, 256, 1, 2, 6, 1>(ctx, p, stream);
}

}  // namespace

namespace {

// Query heads of one row: 16 of them (two column blocks) at most on the tensor
// cores, 8 in fp32 multiply-adds; more are cut into rows of equal size.
void cut_heads(int32_t group, int32_t most, int32_t* chunk, int32_t* n_chunks) {
    *n_chunks = (int32_t)sbt_cdiv(group, most);
    *chunk = (int32_t)sbt_cdiv(group, *n_chunks);
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

// One size for every type: the states of two cut rows per warp, for the
// largest grid, and the descriptors of cut rows.
size_t sbt_paged_attention_workspace_bytes(const sbt_context* ctx, int32_t q_heads, int32_t kv_heads,
                                           int32_t head_dim) {
    int32_t chunk, n;
    cut_heads(q_heads / kv_heads, kAttnMaxHeads, &chunk, &n);
    const size_t g = (size_t)ctx->sm_count * kAttnMaxWarps;
    const size_t heads = chunk <= 8 ? 8 : 16, dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    return round256(g * sizeof(AttnDesc)) + round256(2 * g * kAttnMaxHeads * sizeof(float2)) +
           2 * g * heads * dp * sizeof(float);
}

sbt_status sbt_launch_paged_attention(sbt_context* ctx, sbt_dtype dtype, const SbtHeadRows& q, int32_t batch,
                                      int32_t q_heads, const sbt_kv_cache* cache, const sbt_page_map* map,
                                      const int32_t* seq, float scale, int32_t window, const SbtHeadRows& out,
                                      float* lse, void* workspace, cudaStream_t stream) {
    const int es = sbt_dtype_size(dtype);
    AttnParams p = {};
    p.q = (const char*)q.p, p.k = (const char*)cache->k, p.v = (const char*)cache->v;
    p.out = (char*)const_cast<void*>(out.p), p.lse = lse;
    p.table = map->page_table, p.lens = map->lens, p.seq = seq;
    p.ld_q = q.ld, p.ld_qh = q.ldh, p.ld_out = out.ld, p.ld_oh = out.ldh;
    p.ld_page = cache->ld_page, p.ld_slot = cache->ld_slot, p.ld_head = cache->ld_head;
    p.ld_table = map->ld_table, p.n_pages = map->n_pages;
    p.batch = batch, p.q_heads = q_heads, p.kv_heads = cache->heads, p.group = q_heads / cache->heads;
    cut_heads(p.group, dtype == SBT_F32 ? 8 : kAttnMaxHeads, &p.chunk, &p.n_chunks);
    p.n_seq = map->n_seq, p.head_dim = cache->head_dim, p.window = window;
    const int64_t most = (int64_t)map->max_pages * map->page_size;
    p.max_len = (int32_t)(most < 0x7ffffc00 ? most : 0x7ffffc00);  // tile positions stay below 2^31
    p.page_size = sbt_make_fastdiv((uint32_t)map->page_size);
    p.scale_log2 = scale * 1.4426950408889634f;
    const int64_t bits = (reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) |
                         ((int64_t)p.head_dim | p.ld_page | p.ld_slot | p.ld_head) * es;
    p.copy_bytes = ctx->path == SBT_PATH_SCALAR ? es : bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : es;
    p.q_words = (reinterpret_cast<uintptr_t>(p.q) | ((int64_t)p.head_dim | p.ld_q | p.ld_qh) * es) % 4 == 0;
    p.out_words = (reinterpret_cast<uintptr_t>(p.out) | ((int64_t)p.head_dim | p.ld_out | p.ld_oh) * es) % 4 == 0;
    const size_t g = (size_t)ctx->sm_count * kAttnMaxWarps;
    p.desc = (AttnDesc*)workspace;
    p.part_ml = (float2*)((char*)workspace + round256(g * sizeof(AttnDesc)));
    p.part_o = (float*)((char*)p.part_ml + round256(2 * g * kAttnMaxHeads * sizeof(float2)));
    if (dtype == SBT_F32) return sbt_attention_f32(ctx, p, stream);
    return dtype == SBT_BF16 ? by_dim<true>(ctx, p, stream) : by_dim<false>(ctx, p, stream);
}
