// Paged attention, 32-bit caches: the tile math in fp32 multiply-adds, since a
// tensor-core product would round the operands to fewer bits.
//
// A warp tile is 8 MT positions.  Scores: four lanes share MT positions and take
// every fourth 16-byte piece of their keys; queries are read from shared memory
// (one address per quarter of the warp) once for the MT positions.  Values: a
// lane owns DP / 32 elements of the head and adds p v over the positions.  With
// one or two heads the copies bound the kernel and MT is 1, which leaves room
// for more warps; from three heads on the reads of the query and the shuffles
// do (64 ragged sequences, 64 query heads of 128: 275 us with MT 1).
#include "k_paged_attention.cuh"

namespace {

template <int DP_, int HT, int MT>
struct Fma32 {
    typedef float T;
    static constexpr int ES = 4, TOK = 8 * MT, DP = DP_, HEADS = HT;
    static constexpr int PITCH = DP * 4;
    // scores read four 16-byte pieces of two rows at once: of odd rows the other half of the banks
    static __device__ __forceinline__ int swizzle(int t) { return (t & 1) << 2; }
    static constexpr int EL = DP / 32;         // head elements per lane
    static constexpr int SCRATCH = HT * DP + TOK * HT;  // the query, and a tile's probabilities
    static __device__ __forceinline__ float from_float(float x) { return x; }

    float o[HT][EL];
    float mx[HT], l[HT];

    __device__ __forceinline__ void load_q(const AttnParams& p, const AttnRow& r, int32_t row, float* s_q) {
        const int32_t kvh = row / p.n_chunks, h0 = (row - kvh * p.n_chunks) * p.chunk;
        const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
        const float* base = reinterpret_cast<const float*>(p.q) + r.b * p.ld_q + (kvh * p.group + h0) * p.ld_qh;
        __syncwarp();  // the last tile's reads
        for (int i = threadIdx.x & 31; i < HT * DP; i += 32) {
            const int h = i / DP, d = i - h * DP;
            s_q[i] = h < heads && d < p.head_dim ? sbt_ld(base + h * p.ld_qh + d) : 0.f;
        }
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            mx[h] = -CUDART_INF_F;
            l[h] = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) o[h][e] = 0.f;
        }
        __syncwarp();
    }

    __device__ __forceinline__ void tile(const AttnParams& p, const uint8_t* stage, uint32_t, uint32_t, uint32_t bits,
                                         float* s_q) {
        const int lane = threadIdx.x & 31, t = lane >> 2, part = lane & 3;
        float* const s_p = s_q + HT * DP;
        const uint8_t* const kr = stage + t * PITCH;
        const int k_x = part ^ swizzle(t);  // of rows t and t + 8
        float s[MT][HT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < HT; ++h) s[m][h] = 0.f;
#pragma unroll 4
        for (int i = 0; i < DP / 16; ++i) {
            float4 k4[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m)
                k4[m] = *reinterpret_cast<const float4*>(kr + m * 8 * PITCH + ((i * 4) ^ k_x) * 16);
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                const float4 q4 = *reinterpret_cast<const float4*>(s_q + h * DP + i * 16 + part * 4);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    s[m][h] = fmaf(k4[m].x, q4.x, fmaf(k4[m].y, q4.y, fmaf(k4[m].z, q4.z, fmaf(k4[m].w, q4.w, s[m][h]))));
            }
        }
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            float top = mx[h];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                s[m][h] += __shfl_xor_sync(0xffffffffu, s[m][h], 1);
                s[m][h] += __shfl_xor_sync(0xffffffffu, s[m][h], 2);
                s[m][h] = (bits >> (m * 8 + t)) & 1u ? s[m][h] * p.scale_log2 : -CUDART_INF_F;
                top = fmaxf(top, s[m][h]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float ts = top == -CUDART_INF_F ? 0.f : top;
            const float alpha = sbt_attn::exp2_fast(mx[h] - ts);
            mx[h] = top;
            l[h] *= alpha;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float pr = sbt_attn::exp2_fast(s[m][h] - ts);
                l[h] += pr;  // the four lanes of a position hold the same sum
                if (part == 0) s_p[(m * 8 + t) * HT + h] = pr;
            }
#pragma unroll
            for (int e = 0; e < EL; ++e) o[h][e] *= alpha;
        }
        __syncwarp();
#pragma unroll
        for (int tt = 0; tt < TOK; ++tt) {
            const uint8_t* const vr = stage + (TOK + tt) * PITCH;
            float v[EL], w[HT];
            constexpr int N = EL % 4 == 0 ? 4 : EL % 2 == 0 ? 2 : 1;  // elements per read
#pragma unroll
            for (int e = 0; e < EL; e += N) {
                const int at = lane * EL + e;
                const uint8_t* x = vr + (((at >> 2) ^ swizzle(tt)) << 4) + (at & 3) * 4;
                if (N == 4)
                    *reinterpret_cast<float4*>(v + e) = *reinterpret_cast<const float4*>(x);
                else if (N == 2)
                    *reinterpret_cast<float2*>(v + e) = *reinterpret_cast<const float2*>(x);
                else
                    v[e] = *reinterpret_cast<const float*>(x);
            }
#pragma unroll
            for (int h = 0; h < HT; ++h) w[h] = s_p[tt * HT + h];
#pragma unroll
            for (int h = 0; h < HT; ++h)
#pragma unroll
                for (int e = 0; e < EL; ++e) o[h][e] = fmaf(w[h], v[e], o[h][e]);
        }
        __syncwarp();
    }

    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 4);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 8);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 16);
        }
    }

    __device__ __forceinline__ void put_row(const AttnParams& p, int32_t b, int32_t qh, int32_t heads) {
        finish();
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            if (h >= heads) break;
            const float inv = sbt_attn::inverse(l[h]);
            float* dst = reinterpret_cast<float*>(p.out) + b * p.ld_out + (int64_t)(qh + h) * p.ld_oh;
#pragma unroll
            for (int e = 0; e < EL; ++e)
                if (lane * EL + e < p.head_dim) dst[lane * EL + e] = o[h][e] * inv;
            if (p.lse && lane == 0) p.lse[(int64_t)b * p.q_heads + qh + h] = sbt_attn::log_sum(mx[h], l[h]);
        }
    }

    // the state to dst [DP][HEADS] and ml [HEADS]
    __device__ __forceinline__ void put_part(float* dst, float2* ml) {
        finish();
        const int lane = threadIdx.x & 31;
        dst += lane * EL * HT;
#pragma unroll
        for (int e = 0; e < EL; ++e)
#pragma unroll
            for (int h = 0; h < HT; ++h) dst[e * HT + h] = o[h][e];
        if (lane == 0)
#pragma unroll
            for (int h = 0; h < HT; ++h) ml[h] = make_float2(mx[h], l[h]);
    }
};

// WARPS and BLOCKS with one, WARPS2 and BLOCKS2 with two positions per lane: as many as two stages
// and the query leave room for.
template <int DP, int WARPS, int BLOCKS, int WARPS2, int BLOCKS2>
sbt_status by_heads(sbt_context* ctx, const AttnParams& p, cudaStream_t stream) {
    constexpr int MT = DP <= 128 ? 2 : 1;
    if (p.chunk <= 1) return sbt_attention_enqueue<Fma32<DP, 1, 1>, 2, WARPS, BLOCKS>(ctx, p, stream);
    if (p.chunk <= 2) return sbt_attention_enqueue<Fma32<DP, 2, 1>, 2, WARPS, BLOCKS>(ctx, p, stream);
    if (p.chunk <= 4) return sbt_attention_enqueue<Fma32<DP, 4, MT>, 2, WARPS2, BLOCKS2>(ctx, p, stream);
    return sbt_attention_enqueue<Fma32<DP, 8, MT>, 2, WARPS2, BLOCKS2>(ctx, p, stream);
}

}  // namespace

sbt_status sbt_attention_f32(sbt_context* ctx, const AttnParams& p, cudaStream_t stream) {
    if (p.head_dim <= 64) return by_heads<64, 4, 3, 5, 2>(ctx, p, stream);
    if (p.head_dim <= 96) return by_heads<96, 4, 3, 4, 2>(ctx, p, stream);
    if (p.head_dim <= 128) return by_heads<128, 5, 2, 6, 1>(ctx, p, stream);
    return by_heads<256, 5, 1, 5, 1>(ctx, p, stream);
}
