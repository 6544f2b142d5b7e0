// Attention of one new token per sequence over a paged key-value cache: the
// kernel's skeleton, shared by the 16-bit and the 32-bit translation units.
//
// For a query head with scores s_j = scale * q . k_j over the visible
// positions j, the kernel keeps, one pass over the cache, the running maximum
// m, the sum l = sum_j 2^(s'_j - m) and the vector o = sum_j 2^(s'_j - m) v_j
// (s' = s * log2 e), rescaling l and o by 2^(m_old - m_new) when m grows; all
// three are fp32.  Two such states over disjoint positions join by the same
// rule, which is what lets one row be split over warps and over blocks.
//
// Split.  A row is one (sequence, key-value head, chunk of its query heads).
// Rows are cut into units of 4 warp tiles; all units of all rows lie on one
// line, and block c of G takes the units [c U / G, (c + 1) U / G).  Every block
// so reads the same amount to within one unit whatever the lengths are, and
// the lengths are read on the device.  A row wholly inside one block is
// written by it; of a row cut by block borders each block writes its state to
// the workspace and k_attention_join adds them in block order (the result
// does not depend on which block finished first).
//
// Each warp owns one tile of every unit and a private ring of shared-memory
// stages filled by cp.async, so the main loop has no block-wide barrier; the
// ring runs ahead across row borders, and the warps meet only where a row ends.
// Positions that are masked (past the length, outside the window, on an
// unmapped page) are zero-filled in shared memory and never read from the
// cache, so stale or NaN contents there cannot reach a sum.
#pragma once

#include <math_constants.h>

#include "sbt_internal.cuh"
#include "tc_ptx.cuh"

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnMaxPerSm = 4;    // blocks per SM the workspace is sized for
constexpr int kAttnMaxHeads = 16;   // query heads of one key-value head that one row carries

struct AttnParams {
    const char* q;
    const char* k;
    const char* v;
    char* out;
    float* lse;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* seq;
    int64_t ld_q, ld_qh, ld_out, ld_oh;      // elements
    int64_t ld_page, ld_slot, ld_head;       // elements
    int64_t ld_table, n_pages;
    int32_t batch, q_heads, kv_heads, group; // group: query heads per key-value head
    int32_t chunk, n_chunks;                 // query heads per row, rows per key-value head
    int32_t n_seq, head_dim, window;
    int32_t max_len;                         // max_pages * page_size, capped to int32
    sbt_fastdiv page_size;
    float scale_log2;                        // scale * log2(e)
    int32_t q_words;                         // query rows are read in 4-byte words
    int32_t copy_bytes;                      // 16, 4 or the element size: width of one copy into shared memory
    // workspace
    struct AttnDesc* desc;
    float2* part_ml;                         // [2 G][kAttnMaxHeads] (m, l)
    float* part_o;                           // [2 G][heads][DP]
};

// Row whose first units lie in the block that wrote this and whose last ones
// do not: the parts are slot `first_slot` of block `first` and slot 0 of the
// blocks first + 1 .. last.
struct AttnDesc {
    int32_t valid, b, kvh, chunk;
    int32_t first, last, first_slot, pad;
};

// Visible positions of batch entry b: [lo, hi), and its units.
struct AttnRow {
    int32_t b, seq, lo, hi, base, units;
};

namespace sbt_attn {

template <int UNIT>
__device__ __forceinline__ AttnRow row_of(const AttnParams& p, int32_t b) {
    AttnRow r;
    r.b = b;
    r.seq = p.seq ? __ldg(p.seq + b) : b;
    r.lo = r.hi = r.base = r.units = 0;
    if (r.seq >= 0 && r.seq < p.n_seq) {
        int32_t n = __ldg(p.lens + r.seq);
        n = n < 0 ? 0 : n > p.max_len ? p.max_len : n;
        r.hi = n;
        r.lo = (p.window > 0 && n > p.window) ? n - p.window : 0;
        r.base = r.lo & ~(UNIT - 1);
        r.units = (int32_t)(((int64_t)r.hi - r.base + UNIT - 1) / UNIT);
    }
    return r;
}

__device__ __forceinline__ int64_t range_start(int64_t c, int64_t U, int64_t G) { return c * U / G; }

// Block whose range holds unit u (1 <= G <= U).
__device__ __forceinline__ int32_t block_of(int64_t u, int64_t U, int64_t G) {
    int64_t c = u * G / U;
    while (c + 1 < G && range_start(c + 1, U, G) <= u) ++c;
    while (c > 0 && range_start(c, U, G) > u) --c;
    return (int32_t)c;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sum over the block of one int64 per thread, and its exclusive prefix.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total, int64_t* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) before += s_warp[w];
        sum += s_warp[w];
    }
    *total = sum;
    return before + x - v;
}

}  // namespace sbt_attn

// M is the math of one warp:
//   T, ES         raw element type and its size
//   TOK           positions of one warp tile (a power of two, at most 32)
//   DP            head size padded to what the tile math needs (padding columns are zero)
//   HEADS         query heads a row carries at most
//   PITCH, chunk16(t, c)   bytes between tile rows, place of 16-byte chunk c of row t
//   MERGE_HEADS   heads joined per pass through the merge buffer
//   load_q        query of a row into registers or scratch, state reset (all warps together)
//   tile          one tile; bit t of the mask: position t is visible
//   reduce, put_ml, heads_max, rescale_to, put_o    the state, for the join of the warps
template <class M, int STAGES>
__global__ void __launch_bounds__(kAttnThreads) k_paged_attention(const AttnParams p) {
    using namespace sbt_attn;
    using namespace sbt_ptx;
    constexpr int TOK = M::TOK, DP = M::DP, ES = M::ES, HEADS = M::HEADS, PITCH = M::PITCH;
    constexpr int UNIT = TOK * kAttnWarps;
    constexpr int STAGE_BYTES = 2 * TOK * PITCH;
    constexpr int MERGE_PITCH = DP + 4;  // floats between heads in the merge buffer
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_warp[kAttnWarps];
    __shared__ int64_t s_start[2];       // first unit of the found row's sequence, its batch entry
    __shared__ float s_m[kAttnWarps][HEADS], s_l[kAttnWarps][HEADS];
    __shared__ uint32_t s_mask[kAttnWarps][STAGES];
    float* const s_merge = reinterpret_cast<float*>(smem + (size_t)kAttnWarps * STAGES * STAGE_BYTES);
    float* const s_scratch = s_merge + kAttnWarps * M::MERGE_HEADS * MERGE_PITCH;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t rows_per_seq = p.kv_heads * p.n_chunks;
    uint8_t* const ring = smem + (size_t)warp * STAGES * STAGE_BYTES;
    const uint32_t ring_u32 = smem_u32(ring);

    // the join's blocks may take their places as soon as this grid's are all running
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- units of all rows, and this block's range
    const bool one_scan = p.batch <= kAttnThreads;  // every thread holds its own entry's units
    int64_t total = 0, at = 0;
    int32_t mine = 0;
    if (one_scan) {
        if ((int32_t)threadIdx.x < p.batch) mine = row_of<UNIT>(p, threadIdx.x).units;
        at = block_scan(mine, &total, s_warp);
    } else {
        for (int32_t b = threadIdx.x; b < p.batch; b += kAttnThreads) total += row_of<UNIT>(p, b).units;
        int64_t sum;
        block_scan(total, &sum, s_warp);
        total = sum;
    }
    const int64_t U = total * rows_per_seq;
    const int64_t G = U < gridDim.x ? U : gridDim.x;
    if (threadIdx.x == 0) p.desc[blockIdx.x].valid = 0;

    // rows that see nothing: zeros, and a log-sum-exp of minus infinity
    auto empty_rows = [&]() {
        for (int32_t b = blockIdx.x; b < p.batch; b += gridDim.x) {
            if (row_of<UNIT>(p, b).units != 0) continue;
            for (int32_t i = threadIdx.x; i < p.q_heads * p.head_dim; i += kAttnThreads) {
                const int32_t h = i / p.head_dim, d = i - h * p.head_dim;
                reinterpret_cast<typename M::T*>(p.out)[b * p.ld_out + h * p.ld_oh + d] = M::from_float(0.f);
            }
            if (p.lse)
                for (int32_t h = threadIdx.x; h < p.q_heads; h += kAttnThreads)
                    p.lse[(int64_t)b * p.q_heads + h] = -CUDART_INF_F;
        }
    };
    if (blockIdx.x >= G) {
        empty_rows();
        return;
    }

    const int64_t u0 = range_start(blockIdx.x, U, G), u1 = range_start(blockIdx.x + 1, U, G);

    // ---- the sequence that holds unit u0
    auto claim = [&](int32_t b) {
        if (mine > 0 && at * rows_per_seq <= u0 && u0 < (at + mine) * rows_per_seq) {
            s_start[0] = at * rows_per_seq;
            s_start[1] = b;
        }
    };
    if (one_scan) {
        claim(threadIdx.x);
    } else {
        int64_t before = 0;
        for (int32_t b0 = 0; b0 < p.batch && before * rows_per_seq <= u0; b0 += kAttnThreads) {
            const int32_t b = b0 + threadIdx.x;
            mine = b < p.batch ? row_of<UNIT>(p, b).units : 0;
            int64_t sum;
            at = before + block_scan(mine, &sum, s_warp);
            claim(b);
            before += sum;
        }
    }
    __syncthreads();

    // ---- loader state: runs up to STAGES units ahead of the math
    AttnRow lr = row_of<UNIT>(p, (int32_t)s_start[1]);
    int32_t l_head, l_tile;
    {
        const int64_t in = u0 - s_start[0];
        l_head = (int32_t)(in / lr.units);
        l_tile = (int32_t)(in - (int64_t)l_head * lr.units);
    }
    AttnRow cr = lr;  // math state
    int32_t c_head = l_head, c_tile = l_tile;

    auto next = [&](AttnRow& r, int32_t& head, int32_t& tile) {
        if (++tile < r.units) return;
        tile = 0;
        if (++head < rows_per_seq) return;
        head = 0;
        int32_t b = r.b + 1;
        while (b < p.batch) {
            r = row_of<UNIT>(p, b);
            if (r.units) break;
            ++b;
        }
    };
    // page of this lane's position in the loader's tile (-1: masked), and the position
    auto page_index = [&](int32_t& slot) -> int32_t {
        const int32_t pos = lr.base + l_tile * UNIT + warp * TOK + (lane & (TOK - 1));
        slot = 0;
        if (pos < lr.lo || pos >= lr.hi) return -1;
        const uint32_t pg = sbt_div(p.page_size, (uint32_t)pos);
        slot = pos - (int32_t)(pg * p.page_size.d);
        return __ldg(p.table + (int64_t)lr.seq * p.ld_table + pg);
    };
    auto issue = [&](int stage, int32_t page, int32_t slot, int32_t head) {
        const bool ok = page >= 0 && page < p.n_pages;
        const int32_t kvh = head / p.n_chunks;
        const int64_t off = ok ? (page * p.ld_page + slot * p.ld_slot + kvh * p.ld_head) * ES : -1;
        const uint32_t bits = __ballot_sync(0xffffffffu, ok) & (TOK == 32 ? 0xffffffffu : (1u << (TOK & 31)) - 1u);
        if (lane == 0) s_mask[warp][stage] = bits;
        const uint32_t dst = ring_u32 + stage * STAGE_BYTES;
        if (bits == 0) return;  // the tile is skipped: nothing reads this stage
        if (p.copy_bytes == 16) {
            const int vecs = p.head_dim * ES / 16;   // vectors of one row
            constexpr int LPR = DP * ES / 16 < 32 ? DP * ES / 16 : 32;  // lanes on one row
            constexpr int RPI = 32 / LPR;
            const int c0 = lane % LPR, r0 = lane / LPR;
#pragma unroll
            for (int i = 0; i < TOK / RPI; ++i) {
                const int t = i * RPI + r0;
                const int64_t o = __shfl_sync(0xffffffffu, off, t);
#pragma unroll
                for (int c = c0; c < DP * ES / 16; c += LPR) {
                    if (c < vecs) {
                        const int64_t a = o < 0 ? 0 : o + c * 16;
                        const uint32_t at = t * PITCH + M::chunk16(t, c) * 16;
                        cp_async16(dst + at, p.k + a, o < 0 ? 0 : 16);
                        cp_async16(dst + TOK * PITCH + at, p.v + a, o < 0 ? 0 : 16);
                    }
                }
            }
        } else if (p.copy_bytes == 4) {
            const int words = p.head_dim * ES / 4;
            for (int t = 0; t < TOK; ++t) {
                const int64_t o = __shfl_sync(0xffffffffu, off, t);
                for (int c = lane; c < words; c += 32) {
                    const int64_t a = o < 0 ? 0 : o + c * 4;
                    const uint32_t at = t * PITCH + M::chunk16(t, c / 4) * 16 + (c & 3) * 4;
                    cp_async4(dst + at, p.k + a, o < 0 ? 0 : 4);
                    cp_async4(dst + TOK * PITCH + at, p.v + a, o < 0 ? 0 : 4);
                }
            }
        } else if (ES == 2) {
            typedef typename M::T T;
            uint8_t* const st = ring + stage * STAGE_BYTES;
            constexpr int V = 16 / ES;
            for (int t = 0; t < TOK; ++t) {
                const int64_t o = __shfl_sync(0xffffffffu, off, t);
                for (int c = lane; c < p.head_dim; c += 32) {
                    const int at = t * PITCH + M::chunk16(t, c / V) * 16 + (c % V) * ES;
                    *reinterpret_cast<T*>(st + at) = o < 0 ? T(0) : __ldg(reinterpret_cast<const T*>(p.k + o) + c);
                    *reinterpret_cast<T*>(st + TOK * PITCH + at) =
                        o < 0 ? T(0) : __ldg(reinterpret_cast<const T*>(p.v + o) + c);
                }
            }
        }
    };

    // columns past the head size stay zero for the whole call
    if (p.head_dim < DP) {
        uint32_t* w = reinterpret_cast<uint32_t*>(ring);
        for (int i = lane; i < STAGES * STAGE_BYTES / 4; i += 32) w[i] = 0;
        __syncwarp();
    }

    // the query of a row the loader has reached, towards L2: the math reads it a few units later
    auto prefetch_q = [&](const AttnRow& r, int32_t head) {
        const int32_t kvh = head / p.n_chunks, h0 = (head - kvh * p.n_chunks) * p.chunk;
        const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
        if (lane >= heads) return;
        const char* x = p.q + (r.b * p.ld_q + (int64_t)(kvh * p.group + h0 + lane) * p.ld_qh) * ES;
        for (int i = 0; i < p.head_dim * ES; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + i));
    };

    int64_t l_u = u0;
    int32_t slot_next, page_next = page_index(slot_next);
    auto load_step = [&](int stage) {  // issue the loader's unit, then look up the next one's pages
        if (l_u < u1) {
            issue(stage, page_next, slot_next, l_head);
            if (++l_u < u1) {
                next(lr, l_head, l_tile);
                page_next = page_index(slot_next);
                if (l_tile == 0 && warp == 0) prefetch_q(lr, l_head);
            }
        }
        cp_commit();
    };
#pragma unroll 1
    for (int s = 0; s < STAGES - 1; ++s) load_step(s);

    M m;
    m.load_q(p, cr, c_head, s_scratch);
    int stage = 0;
    int64_t row_u0 = u0 - c_tile;  // first unit of the current row on the line
    bool row_cut = c_tile != 0;    // the row began in an earlier block
    for (int64_t u = u0; u < u1; ++u) {
        cp_wait<STAGES - 2>();
        __syncwarp();
        // the stage read in the last step is free: refill it before this step's math
        load_step(stage == 0 ? STAGES - 1 : stage - 1);
        const uint32_t bits = s_mask[warp][stage];
        if (bits) {
            const uint32_t k_s = ring_u32 + stage * STAGE_BYTES;
            m.tile(p, ring + stage * STAGE_BYTES, k_s, k_s + TOK * PITCH, bits, s_scratch);
        }
        stage = stage + 1 == STAGES ? 0 : stage + 1;

        const bool row_end = c_tile + 1 == cr.units;
        if (row_end || u + 1 == u1) {
            // ---- join the four warps
            m.reduce();
            m.put_ml(s_m[warp], s_l[warp]);
            __syncthreads();
            float top[M::OWN], own[M::OWN];
            m.heads_max(s_m, top);
#pragma unroll
            for (int i = 0; i < M::OWN; ++i) own[i] = top[i] == -CUDART_INF_F ? 0.f : top[i];
            m.rescale_to(own);
            const int32_t kvh = c_head / p.n_chunks, chunk = c_head - kvh * p.n_chunks;
            const bool whole = row_end && !row_cut;
            const int part_slot = row_cut || row_u0 == u0 ? 0 : 1;
            const int32_t h0 = chunk * p.chunk;
            const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
            constexpr int HB = M::MERGE_HEADS;  // heads per pass through the merge buffer
#pragma unroll
            for (int hb = 0; hb < HEADS; hb += HB) {
                if (hb >= heads) break;
                m.put_o(s_merge + (size_t)warp * HB * MERGE_PITCH, MERGE_PITCH, hb);
                __syncthreads();
                for (int i = threadIdx.x; i < HB * (DP / 4); i += kAttnThreads) {
                    const int h = i / (DP / 4), d = (i - h * (DP / 4)) * 4, head = hb + h;
                    if (head >= heads) break;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    float mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll
                    for (int w = 0; w < kAttnWarps; ++w) mm = fmaxf(mm, s_m[w][head]);
                    const float ms = mm == -CUDART_INF_F ? 0.f : mm;
#pragma unroll
                    for (int w = 0; w < kAttnWarps; ++w) {
                        const float4 x = *reinterpret_cast<const float4*>(s_merge + ((size_t)w * HB + h) * MERGE_PITCH + d);
                        o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
                        ll += s_l[w][head] * exp2_fast(s_m[w][head] - ms);
                    }
                    const int32_t qh = kvh * p.group + h0 + head;
                    if (whole) {
                        const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
                        typename M::T* dst =
                            reinterpret_cast<typename M::T*>(p.out) + cr.b * p.ld_out + qh * p.ld_oh + d;
                        if (d + 0 < p.head_dim) dst[0] = M::from_float(o.x * inv);
                        if (d + 1 < p.head_dim) dst[1] = M::from_float(o.y * inv);
                        if (d + 2 < p.head_dim) dst[2] = M::from_float(o.z * inv);
                        if (d + 3 < p.head_dim) dst[3] = M::from_float(o.w * inv);
                        if (d == 0 && p.lse)
                            p.lse[(int64_t)cr.b * p.q_heads + qh] =
                                ll == 0.f ? -CUDART_INF_F : (mm + log2f(ll)) * 0.6931471805599453f;
                    } else {
                        const int64_t s = 2 * (int64_t)blockIdx.x + part_slot;
                        *reinterpret_cast<float4*>(p.part_o + (s * HEADS + head) * DP + d) = o;
                        if (d == 0) p.part_ml[s * kAttnMaxHeads + head] = make_float2(mm, ll);
                    }
                }
                __syncthreads();
            }
            if (!whole && !row_cut && threadIdx.x == 0) {
                AttnDesc e;
                e.valid = 1, e.b = cr.b, e.kvh = kvh, e.chunk = chunk;
                e.first = blockIdx.x;
                e.last = block_of(row_u0 + cr.units - 1, U, G);
                e.first_slot = part_slot;
                e.pad = 0;
                p.desc[blockIdx.x] = e;
            }
            if (u + 1 < u1) {
                row_u0 = u + 1;
                row_cut = false;
                next(cr, c_head, c_tile);
                m.load_q(p, cr, c_head, s_scratch);
            }
        } else {
            ++c_tile;
        }
    }
    empty_rows();
}

// Joins the parts of the rows that block borders cut, in block order.  Block
// (c, y) looks at the row that began in block c, if one did.  Up to
// kJoinFew parts (rows are many): blocks with y % 8 == 0 give a warp to each of
// eight heads.  More parts (rows are few): block y takes head y, its
// eight warps the parts in turn, and the warps meet in shared memory.
constexpr int kJoinFew = 64;

template <class T, T (*FROM)(float), int HEADS, int DP>
__global__ void __launch_bounds__(256) k_attention_join(const AttnParams p) {
    using namespace sbt_attn;
    constexpr int NV = (DP + 127) / 128;  // float4s of a head per lane
    __shared__ float s_l[8];
    __shared__ float4 s_o[8][NV][32];
    sbt_ptx::griddep_wait();
    const AttnDesc e = p.desc[blockIdx.x];
    if (!e.valid) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = e.last - e.first + 1;
    const bool few = n <= kJoinFew;
    if (few && (blockIdx.y & 7)) return;
    const int32_t h0 = e.chunk * p.chunk;
    const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
    const int head = few ? blockIdx.y + warp : blockIdx.y;
    const int i0 = few ? 0 : warp, di = few ? 1 : 8;
    if (head >= heads) return;  // the whole block, unless each warp is by itself
    auto slot = [&](int i) -> int64_t { return 2 * (int64_t)(e.first + i) + (i == 0 ? e.first_slot : 0); };

    float mm = -CUDART_INF_F;
    for (int i = lane; i < n; i += 32) mm = fmaxf(mm, p.part_ml[slot(i) * kAttnMaxHeads + head].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
    const float ms = mm == -CUDART_INF_F ? 0.f : mm;

    float4 o[NV];
    float l = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = i0; i < n; i += di) {
        const int64_t s = slot(i);
        const float2 ml = p.part_ml[s * kAttnMaxHeads + head];
        const float w = exp2_fast(ml.x - ms);
        l += ml.y * w;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int d = v * 128 + lane * 4;
            if (d < DP) {
                const float4 x = *reinterpret_cast<const float4*>(p.part_o + (s * HEADS + head) * DP + d);
                o[v].x += x.x * w, o[v].y += x.y * w, o[v].z += x.z * w, o[v].w += x.w * w;
            }
        }
    }
    if (!few) {
#pragma unroll
        for (int v = 0; v < NV; ++v) s_o[warp][v][lane] = o[v];
        if (lane == 0) s_l[warp] = l;
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int w = 1; w < 8; ++w) {
            l += s_l[w];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const float4 x = s_o[w][v][lane];
                o[v].x += x.x, o[v].y += x.y, o[v].z += x.z, o[v].w += x.w;
            }
        }
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int32_t qh = e.kvh * p.group + h0 + head;
    T* const dst = reinterpret_cast<T*>(p.out) + e.b * p.ld_out + qh * p.ld_oh;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int d = v * 128 + lane * 4;
        if (d + 0 < p.head_dim) dst[d + 0] = FROM(o[v].x * inv);
        if (d + 1 < p.head_dim) dst[d + 1] = FROM(o[v].y * inv);
        if (d + 2 < p.head_dim) dst[d + 2] = FROM(o[v].z * inv);
        if (d + 3 < p.head_dim) dst[d + 3] = FROM(o[v].w * inv);
    }
    if (lane == 0 && p.lse)
        p.lse[(int64_t)e.b * p.q_heads + qh] = l == 0.f ? -CUDART_INF_F : (mm + log2f(l)) * 0.6931471805599453f;
}

// Enqueues the kernel and the join for one instantiation.
template <class M, int STAGES>
sbt_status sbt_attention_enqueue(sbt_context* ctx, const AttnParams& p, cudaStream_t stream) {
    constexpr int HB = M::MERGE_HEADS;
    constexpr size_t smem = (size_t)kAttnWarps * STAGES * 2 * M::TOK * M::PITCH +
                            (size_t)kAttnWarps * HB * (M::DP + 4) * sizeof(float) + M::SCRATCH_BYTES;
    sbt_status st;
    int grid = sbt_resident_blocks<k_paged_attention<M, STAGES>>(ctx, kAttnThreads, smem);
    if (grid > ctx->sm_count * kAttnMaxPerSm) grid = ctx->sm_count * kAttnMaxPerSm;
    k_paged_attention<M, STAGES><<<grid, kAttnThreads, smem, stream>>>(p);
    if ((st = sbt_after_launch(ctx, "paged_attention"))) return st;
    const int heads = p.group < p.chunk ? p.group : p.chunk;
    if ((st = sbt_cuda_check(sbt_launch_dependent(k_attention_join<typename M::T, M::from_float, M::HEADS, M::DP>,
                                                  dim3(grid, heads), dim3(256), 0, stream, p),
                             "paged_attention join launch")))
        return st;
    return sbt_after_launch(ctx, "paged_attention join");
}

sbt_status sbt_attention_f32(sbt_context* ctx, const AttnParams& p, cudaStream_t stream);
