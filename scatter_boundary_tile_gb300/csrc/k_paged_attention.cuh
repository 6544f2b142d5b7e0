// Attention of one new token per sequence over a paged key-value cache: the
// kernel's skeleton, shared by the 16-bit and the 32-bit translation units.
//
// For a query head with scores s_j = scale * q . k_j over the visible
// positions j, the kernel keeps, one pass over the cache, the running maximum
// m, the sum l = sum_j 2^(s'_j - m) and the vector o = sum_j 2^(s'_j - m) v_j
// (s' = s * log2 e), rescaling l and o by 2^(m_old - m_new) when m grows; all
// three are fp32.  Two such states over disjoint positions join by the same
// rule, which is what lets one row be split.
//
// Split.  A row is one (sequence, key-value head, chunk of its query heads),
// cut into tiles of TOK positions.  All rows lie on one line, each as kRowCost
// empty places (what starting and ending a row costs, in tiles) and a place per
// tile; warp c of G takes the tiles at U / G of the U places, in order.  So
// every warp has the same work whatever the lengths are, and the lengths are
// read on the device.  A row wholly inside one warp's range is written by that
// warp; of a row cut by range borders each warp writes its state to the
// workspace and k_attention_join adds them in the order of the line (the result
// does not depend on which warp finished first).
//
// After the first prefix sum no warp waits for another: each has a private ring
// of shared-memory stages filled by cp.async, which runs ahead of the math and
// across row ends.  Measured before it, bf16, 32 query and 8 key-value heads of
// 128: ranges per block with a join of its warps at each row end, 103 us on 64
// ragged sequences up to 4096 and 142 us on 1024 up to 128 (now 94-97 and 68);
// rows fetched by the bulk-copy engine, one 256-byte row a lane, 136 us on the
// former: the engine starts about one row per 15 cycles.
//
// Positions that are masked (past the length, outside the window, on an
// unmapped page) are never read from the cache and are zero in shared memory,
// so stale or NaN contents there cannot reach a sum.
#pragma once

#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>

#include "sbt_internal.cuh"
#include "tc_ptx.cuh"

constexpr int kAttnMaxWarps = 16;   // warps per SM the workspace is sized for
constexpr int kClusterMost = 8, kClusterTiles = 16;
// 1024 sequences up to 128: 98 us at 0, 68 at 2 and 3, 70 at 5; 64 up to 4096: the same at all four.
constexpr int kRowCost = 3;
constexpr int kAttnMaxHeads = 16;   // query heads of one key-value head that one row carries

// A cut row: the warps first .. last hold its parts, in slot 2 first +
// first_slot and in slots 2 c of the others -- except that a block which lies
// wholly inside the row has joined its warps' parts in its first warp's slot.
// That holds for all blocks between the first's and the last's, and for those
// two as the flags say.
struct AttnDesc {
    int32_t valid, b, kvh, chunk;
    int32_t first, last, first_slot, joined;  // joined: bit 0 the first's block, bit 1 the last's
};

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
    int32_t q_words, out_words;              // rows of q / out start on 4 bytes and head_dim fills whole words
    int32_t tile_in_page;                    // pages hold whole tiles
    int32_t copy_bytes;                      // 16, 8, 4 or the element size: width of one copy into shared memory
    int32_t cluster;                         // blocks per row of the cluster form
    int32_t desc_by_row;                     // descriptors by row (there are no more rows than warps), else by warp
    // workspace
    AttnDesc* desc;
    float2* part_ml;                         // [2 G][HEADS] (m, l)
    float* part_o;                           // [2 G][DP][HEADS]
};

// Visible positions of batch entry b: [lo, hi), and its tiles from `base` on.
struct AttnRow {
    int32_t b, seq, lo, hi, base, tiles;
};

namespace sbt_attn {

template <int TOK>
__device__ __forceinline__ AttnRow row_of(const AttnParams& p, int32_t b) {
    AttnRow r;
    r.b = b;
    r.seq = p.seq ? sbt_ld(p.seq + b) : b;
    r.lo = r.hi = r.base = r.tiles = 0;
    if (r.seq >= 0 && r.seq < p.n_seq) {
        int32_t n = sbt_ld(p.lens + r.seq);
        n = n < 0 ? 0 : n > p.max_len ? p.max_len : n;
        r.hi = n;
        r.lo = (p.window > 0 && n > p.window) ? n - p.window : 0;
        r.base = r.lo & ~(TOK - 1);
        r.tiles = (r.hi - r.base + TOK - 1) / TOK;
    }
    return r;
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // a >= 0, b > 0
    return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// U places over G warps (1 <= G <= U): the first `more` warps take size + 1, the others size.
struct Line {
    int64_t size, more;
    __device__ __forceinline__ Line(int64_t U, int64_t G) : size(divide(U, G)) { more = U - size * G; }
    __device__ __forceinline__ int64_t start(int64_t c) const { return c * size + (c < more ? c : more); }
    // warp whose range holds place u
    __device__ __forceinline__ int32_t warp_of(int64_t u) const {
        const int64_t big = more * (size + 1);
        return (int32_t)(u < big ? divide(u, size + 1) : more + divide(u - big, size));
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
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

// 1 / l, or 0 for a row that saw nothing (l = 0); NaN stays NaN.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
}

// Exclusive prefix over the block of one int64 per thread, and the sum.
template <int WARPS>
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
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += s_warp[w];
        sum += s_warp[w];
    }
    *total = sum;
    return before + x - v;
}

}  // namespace sbt_attn

// M is the math of one warp:
//   T, ES         raw element type and its size
//   TOK           positions of one tile (a power of two, at most 32)
//   DP            head size padded to what the tile math needs (padding columns are zero)
//   HEADS         query heads a row carries at most (a power of two)
//   PITCH         bytes between tile rows
//   swizzle(t)    what the 16-byte chunk numbers of row t are XORed with.  Rows start on 64 bytes
//                 or more: a copy whose global lines straddle shared-memory lines asks L2 twice
//                 (rows padded by 16 bytes: 39 % of the sectors, 105 us against 98 on 64 ragged
//                 sequences); the XOR keeps the math's reads free of bank conflicts
//   SCRATCH       floats of shared memory per warp
//   load_q        query of a row into registers or scratch, state reset
//   tile          one tile; bit t of the mask: position t is visible
//   put_row       the finished row to out and lse
//   put_part      the state to memory

// One warp's tiles on their way into its ring: the loads run STAGES - 1 tiles
// ahead of the math and cross row ends by themselves.
template <class M, int STAGES>
struct AttnLoader {
    static constexpr int TOK = M::TOK, DP = M::DP, ES = M::ES, PITCH = M::PITCH;
    static constexpr int STAGE_BYTES = 2 * TOK * PITCH;
    static constexpr uint32_t ALL = TOK == 32 ? 0xffffffffu : (1u << (TOK & 31)) - 1u;
    // 16-byte copies: LPR lanes on one row, RPI rows at a time
    static constexpr int VECS = DP * ES / 16, LPR = VECS > 16 ? 32 : VECS > 8 ? 16 : 8, RPI = 32 / LPR;

    const AttnParams& p;
    uint8_t* const ring;
    uint32_t* const mask;   // [STAGES] visible positions of each stage's tile
    const uint32_t ring_u32;
    const int lane, c0, r0, vecs;
    const int32_t rows_per_seq;
    const int64_t v_minus_k;
    AttnRow row;
    int32_t head, tile;
    int64_t at;             // the next tile's place on the line
    const int64_t end;      // of the warp's range
    int32_t page, slot;     // this lane's position in the next tile: its page (-1: masked) and slot

    // the tiles at the places [at, end) of the line, the first of which is tile `tile` of row (row, head)
    __device__ __forceinline__ AttnLoader(const AttnParams& p_, uint8_t* ring_, uint32_t* mask_, const AttnRow& row_,
                                          int32_t head_, int32_t tile_, int64_t at_, int64_t end_)
        : p(p_), ring(ring_), mask(mask_), ring_u32(sbt_ptx::smem_u32(ring_)), lane(threadIdx.x & 31),
          c0((threadIdx.x & 31) % LPR), r0((threadIdx.x & 31) / LPR), vecs(p_.head_dim * ES / 16),
          rows_per_seq(p_.kv_heads * p_.n_chunks), v_minus_k(p_.v - p_.k), row(row_), head(head_), tile(tile_),
          at(at_), end(end_) {
        // columns past the head size stay zero for the whole call
        if (p.head_dim < DP) {
            uint32_t* w = reinterpret_cast<uint32_t*>(ring);
            for (int i = lane; i < STAGES * STAGE_BYTES / 4; i += 32) w[i] = 0;
            __syncwarp();
        }
        look_up();
#pragma unroll 1
        for (int s = 0; s < STAGES - 1; ++s) step(s);
    }

    // The tile after (r, h, t) at place u.
    __device__ __forceinline__ void next(AttnRow& r, int32_t& h, int32_t& t, int64_t& u) const {
        ++u;
        if (++t < r.tiles) return;
        t = 0;
        u += kRowCost;
        if (u >= end) return;  // the range ends here
        if (++h < rows_per_seq) return;
        h = 0;
        int32_t b = r.b + 1;
        while (b < p.batch) {
            r = sbt_attn::row_of<TOK>(p, b);
            if (r.tiles) break;
            ++b;
        }
    }

    __device__ __forceinline__ void look_up() {
        const int32_t pos = row.base + tile * TOK + (lane & (TOK - 1));
        slot = 0, page = -1;
        if (at >= end || pos < row.lo || pos >= row.hi) return;
        const uint32_t pg = sbt_div(p.page_size, (uint32_t)pos);
        slot = pos - (int32_t)(pg * p.page_size.d);
        page = sbt_ld(p.table + (int64_t)row.seq * p.ld_table + pg);
    }

    // The query of a row, towards L2: the math reads it a tile or two later.
    __device__ __forceinline__ void prefetch_q() const {
        const int32_t kvh = head / p.n_chunks, h0 = (head - kvh * p.n_chunks) * p.chunk;
        const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
        if (lane >= heads) return;
        const char* x = p.q + (row.b * p.ld_q + (int64_t)(kvh * p.group + h0 + lane) * p.ld_qh) * ES;
        for (int i = 0; i < p.head_dim * ES; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + i));
    }

    // Starts the next tile's copies into `stage`, then looks up the pages of the one after.
    __device__ __forceinline__ void step(int stage) {
        if (at < end) {
            issue(stage);
            next(row, head, tile, at);
            if (tile == 0 && at < end) prefetch_q();
            look_up();
        }
        sbt_attn::cp_commit();
    }

    __device__ __forceinline__ void issue(int stage) {
        using namespace sbt_attn;
        const bool ok = page >= 0 && page < p.n_pages;
        const int32_t kvh = p.n_chunks == 1 ? head : head / p.n_chunks;
        const int64_t off = ok ? (page * p.ld_page + slot * p.ld_slot + kvh * p.ld_head) * ES : -1;
        const uint32_t bits = __ballot_sync(0xffffffffu, ok) & ALL;
        if (lane == 0) mask[stage] = bits;
        const uint32_t dst = ring_u32 + stage * STAGE_BYTES;
        if (bits == 0) return;  // the tile is skipped: nothing reads this stage
        if (p.copy_bytes == 16) {
            // place of row i RPI + r0, vector v + c0, relative to the stage
            auto place = [&](int i, int v) -> uint32_t {
                const int t = i * RPI + r0;
                return t * PITCH + (((v + c0) ^ M::swizzle(t)) << 4);
            };
            if (p.tile_in_page && bits == ALL) {
                // every row of the tile follows the first at the slots' stride
                const char* k = p.k + __shfl_sync(0xffffffffu, off, 0) + r0 * (p.ld_slot * ES) + c0 * 16;
                const int64_t step = RPI * p.ld_slot * ES;
#pragma unroll
                for (int i = 0; i < TOK / RPI; ++i) {
#pragma unroll
                    for (int v = 0; v < VECS; v += LPR)
                        if (c0 + v < vecs) {
                            cp_async16(dst + place(i, v), k + v * 16, 16);
                            cp_async16(dst + TOK * PITCH + place(i, v), k + v_minus_k + v * 16, 16);
                        }
                    k += step;
                }
            } else {
#pragma unroll
                for (int i = 0; i < TOK / RPI; ++i) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, i * RPI + r0);
                    const char* k = p.k + (o < 0 ? 0 : o) + c0 * 16;
                    const int n = o < 0 ? 0 : 16;  // no byte is read of a masked row: zeros
#pragma unroll
                    for (int v = 0; v < VECS; v += LPR)
                        if (c0 + v < vecs) {
                            cp_async16(dst + place(i, v), k + v * 16, n);
                            cp_async16(dst + TOK * PITCH + place(i, v), k + v_minus_k + v * 16, n);
                        }
                }
            }
        } else if (p.copy_bytes == 8) {
            // 64 sequences up to 4096 at head size 100: 142 us, 154 in words of 4 bytes
            const int pairs = p.head_dim * ES / 8;
            for (int t = 0; t < TOK; ++t) {
                const int64_t o = __shfl_sync(0xffffffffu, off, t);
                for (int w = lane; w < pairs; w += 32) {
                    const int64_t a = o < 0 ? 0 : o + w * 8;
                    const uint32_t s = t * PITCH + (((w >> 1) ^ M::swizzle(t)) << 4) + (w & 1) * 8;
                    cp_async8(dst + s, p.k + a, o < 0 ? 0 : 8);
                    cp_async8(dst + TOK * PITCH + s, p.v + a, o < 0 ? 0 : 8);
                }
            }
        } else if (p.copy_bytes == 4) {
            const int words = p.head_dim * ES / 4;
            for (int t = 0; t < TOK; ++t) {
                const int64_t o = __shfl_sync(0xffffffffu, off, t);
                for (int w = lane; w < words; w += 32) {
                    const int64_t a = o < 0 ? 0 : o + w * 4;
                    const uint32_t s = t * PITCH + (((w >> 2) ^ M::swizzle(t)) << 4) + (w & 3) * 4;
                    cp_async4(dst + s, p.k + a, o < 0 ? 0 : 4);
                    cp_async4(dst + TOK * PITCH + s, p.v + a, o < 0 ? 0 : 4);
                }
            }
        } else if (ES == 2) {
            typedef typename M::T T;
            uint8_t* const st = ring + stage * STAGE_BYTES;
            for (int t = 0; t < TOK; ++t) {
                const int64_t o = __shfl_sync(0xffffffffu, off, t);
                for (int e = lane; e < p.head_dim; e += 32) {
                    const int a = t * PITCH + (((e >> 3) ^ M::swizzle(t)) << 4) + (e & 7) * ES;
                    *reinterpret_cast<T*>(st + a) = o < 0 ? T(0) : sbt_ld(reinterpret_cast<const T*>(p.k + o) + e);
                    *reinterpret_cast<T*>(st + TOK * PITCH + a) =
                        o < 0 ? T(0) : sbt_ld(reinterpret_cast<const T*>(p.v + o) + e);
                }
            }
        }
    }

    // Waits for the tile in `stage`, refills the stage the last step read, and does the math.
    __device__ __forceinline__ void do_tile(M& m, int& stage, float* scratch) {
        sbt_attn::cp_wait<STAGES - 2>();
        __syncwarp();
        step(stage == 0 ? STAGES - 1 : stage - 1);
        const uint32_t bits = mask[stage];
        if (bits) {
            const uint32_t k_s = ring_u32 + stage * STAGE_BYTES;
            m.tile(p, ring + stage * STAGE_BYTES, k_s, k_s + TOK * PITCH, bits, scratch);
        }
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
};

// (m, l) of head h over `n` states, and each state's weight for element i of o.
template <class M>
__device__ __forceinline__ float attn_join(const float* o, const float2* ml, int64_t o_step, int ml_step, int n, int i,
                                           float* top_out, float* l_out) {
    const int h = i % M::HEADS;
    float top = -CUDART_INF_F, l = 0.f, x = 0.f;
    for (int w = 0; w < n; ++w) top = fmaxf(top, ml[w * ml_step + h].x);
    const float ts = top == -CUDART_INF_F ? 0.f : top;
    for (int w = 0; w < n; ++w) {
        const float2 v = ml[w * ml_step + h];
        const float a = sbt_attn::exp2_fast(v.x - ts);
        l += v.y * a;
        x += o[w * o_step + i] * a;
    }
    *top_out = top, *l_out = l;
    return x;
}

template <class M, int STAGES, int WARPS, int BLOCKS>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS) k_paged_attention(const AttnParams p) {
    using namespace sbt_attn;
    typedef AttnLoader<M, STAGES> Loader;
    constexpr int TOK = M::TOK, DP = M::DP, THREADS = 32 * WARPS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_warp[WARPS];
    __shared__ int64_t s_first[THREADS];  // first tile of each batch entry of a scan step
    __shared__ uint32_t s_mask[WARPS][STAGES];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t rows_per_seq = p.kv_heads * p.n_chunks;
    float* const scratch =
        reinterpret_cast<float*>(smem + (size_t)WARPS * STAGES * Loader::STAGE_BYTES) + (size_t)warp * M::SCRATCH;
    sbt_ptx::griddep_wait();

    // ---- the line: places of all rows (of one row of entry b: its tiles and kRowCost, or none)
    auto places = [&](int32_t b) {
        const int32_t n = row_of<TOK>(p, b).tiles;
        return n ? n + kRowCost : 0;
    };
    const bool one_step = p.batch <= THREADS;  // every thread holds its own entry's places
    int64_t total = 0, at = 0;
    int32_t mine = 0;
    if (one_step) {
        if ((int32_t)threadIdx.x < p.batch) mine = places(threadIdx.x);
        at = block_scan<WARPS>(mine, &total, s_warp);
    } else {
        for (uint32_t b = threadIdx.x; b < (uint32_t)p.batch; b += THREADS) total += places((int32_t)b);
        int64_t sum;
        block_scan<WARPS>(total, &sum, s_warp);
        total = sum;
    }
    const int64_t U = total * rows_per_seq;
    const int64_t all_warps = (int64_t)gridDim.x * WARPS, G = U < all_warps ? U : all_warps;
    const int64_t c = (int64_t)blockIdx.x * WARPS + warp;
    bool idle = c >= G;
    const Line line(U, G > 0 ? G : 1);
    const int64_t u0 = idle ? U : line.start(c), u1 = idle ? U : line.start(c + 1);

    // ---- the batch entry that holds place u0, and its first place
    int32_t b_first = 0;
    int64_t u_first = 0;
    {
        int64_t before = 0;
        for (uint32_t b0 = 0; b0 < (uint32_t)p.batch; b0 += THREADS) {  // unsigned: the last step may pass 2^31
            int64_t sum = total;
            if (!one_step) {
                const uint32_t b = b0 + threadIdx.x;
                mine = b < (uint32_t)p.batch ? places((int32_t)b) : 0;
                at = before + block_scan<WARPS>(mine, &sum, s_warp);
            }
            s_first[threadIdx.x] = at * rows_per_seq;
            __syncthreads();
            if (!idle && before * rows_per_seq <= u0 && u0 < (before + sum) * rows_per_seq) {
                for (int i = lane; i < THREADS; i += 32) {
                    const int64_t end = i + 1 < THREADS ? s_first[i + 1] : (before + sum) * rows_per_seq;
                    const uint32_t hit = __ballot_sync(0xffffffffu, s_first[i] <= u0 && u0 < end);
                    if (hit) {
                        b_first = (int32_t)b0 + (i & ~31) + __ffs(hit) - 1;
                        u_first = s_first[(i & ~31) + __ffs(hit) - 1];
                    }
                }
            }
            __syncthreads();
            before += sum;
        }
    }

    // ---- rows that see nothing: zeros, and a log-sum-exp of minus infinity
    auto empty_rows = [&]() {
        for (int64_t b = c; b < p.batch; b += all_warps) {
            if (row_of<TOK>(p, (int32_t)b).tiles != 0) continue;
            for (uint32_t i = lane; i < (uint32_t)(p.q_heads * p.head_dim); i += 32) {
                const uint32_t h = i / (uint32_t)p.head_dim, d = i - h * (uint32_t)p.head_dim;
                reinterpret_cast<typename M::T*>(p.out)[b * p.ld_out + h * p.ld_oh + d] = typename M::T(0);
            }
            if (p.lse)
                for (uint32_t h = lane; h < (uint32_t)p.q_heads; h += 32) p.lse[b * p.q_heads + h] = -CUDART_INF_F;
            if (p.desc_by_row)
                for (uint32_t h = lane; h < (uint32_t)rows_per_seq; h += 32) p.desc[b * rows_per_seq + h].valid = 0;
        }
    };
    if (!p.desc_by_row && lane == 0) p.desc[c].valid = 0;

    // ---- this warp's tiles
    AttnRow cr;
    int32_t c_head = 0, c_tile = 0;
    int64_t at_u = 0;  // place of the tile the math is at
    if (!idle) {
        cr = row_of<TOK>(p, b_first);
        const int64_t width = cr.tiles + kRowCost;
        c_head = (int32_t)divide(u0 - u_first, width);
        const int64_t row_u = u_first + c_head * width + kRowCost;
        at_u = u0 > row_u ? u0 : row_u;
        c_tile = (int32_t)(at_u - row_u);
        idle = at_u >= u1;  // nothing but a row's empty places
    }
    if (idle) {
        empty_rows();
        return;
    }
    Loader loader(p, smem + (size_t)warp * STAGES * Loader::STAGE_BYTES, s_mask[warp], cr, c_head, c_tile, at_u, u1);

    // block B's ranges lie wholly inside a row whose tiles are at the places [a, e)
    auto inside = [&](int64_t B, int64_t a, int64_t e) {
        return (B + 1) * WARPS <= G && a <= line.start(B * WARPS) && e >= line.start((B + 1) * WARPS);
    };

    M m;
    m.load_q(p, cr, c_head, scratch);
    int stage = 0;
    bool first = true;           // the current row is the range's first
    bool cut = c_tile != 0;      // it began in an earlier range
    bool join_block = false;     // this block's warps join their parts
    bool more = true;
#pragma unroll 1
    while (more) {
        loader.do_tile(m, stage, scratch);
        const bool row_end = c_tile + 1 == cr.tiles;
        more = at_u + (row_end ? 1 + kRowCost : 1) < u1;
        if (!row_end && more) {
            ++c_tile;
            ++at_u;
            continue;
        }
        const int32_t kvh = c_head / p.n_chunks, chunk = c_head - kvh * p.n_chunks, h0 = chunk * p.chunk;
        const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk, qh = kvh * p.group + h0;
        AttnDesc e;
        e.valid = 0;
        if (row_end && !cut) {
            m.put_row(p, cr.b, qh, heads);
        } else {
            const int slot = first ? 0 : 1;
            const int64_t row_a = at_u - c_tile, row_e = row_a + cr.tiles;  // the row's tiles on the line
            join_block = first && !more && inside(blockIdx.x, row_a, row_e);
            if (!join_block)
                m.put_part(p.part_o + (2 * c + slot) * M::HEADS * DP, p.part_ml + (2 * c + slot) * M::HEADS);
            if (!cut) {
                e.valid = 1, e.b = cr.b, e.kvh = kvh, e.chunk = chunk;
                e.first = (int32_t)c, e.first_slot = slot;
                e.last = line.warp_of(row_e - 1);
                e.joined = (inside(blockIdx.x, row_a, row_e) ? 1 : 0) | (inside(e.last / WARPS, row_a, row_e) ? 2 : 0);
            }
        }
        if (!cut && lane == 0) {
            if (p.desc_by_row)
                p.desc[(int64_t)cr.b * rows_per_seq + c_head] = e;
            else if (e.valid)
                p.desc[c] = e;
        }
        if (more) {
            first = cut = false;
            loader.next(cr, c_head, c_tile, at_u);
            m.load_q(p, cr, c_head, scratch);
        }
    }
    if (join_block) {  // the same for all warps of the block; the ring is free
        constexpr int N = M::HEADS * DP;
        float* const s_o = reinterpret_cast<float*>(smem);
        float2* const s_ml = reinterpret_cast<float2*>(s_o + WARPS * N);
        cp_wait<0>();
        __syncthreads();
        m.put_part(s_o + warp * N, s_ml + warp * M::HEADS);
        __syncthreads();
        const int64_t slot = 2 * (int64_t)blockIdx.x * WARPS;
        for (int i = threadIdx.x; i < N; i += THREADS) {
            float top, l;
            p.part_o[slot * N + i] = attn_join<M>(s_o, s_ml, N, M::HEADS, WARPS, i, &top, &l);
            if (i < M::HEADS) p.part_ml[slot * M::HEADS + i] = make_float2(top, l);
        }
    }
    empty_rows();
}

// Few rows that are not long: a cluster of p.cluster blocks per row, whose warps
// take its tiles evenly and join their states through distributed shared
// memory.  One launch, no workspace and no prefix sum; but a long row has only
// one cluster's warps.
template <class M, int STAGES, int WARPS, int BLOCKS>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS) k_paged_attention_cluster(const AttnParams p) {
    using namespace sbt_attn;
    namespace cg = cooperative_groups;
    typedef AttnLoader<M, STAGES> Loader;
    constexpr int N = M::HEADS * M::DP, THREADS = 32 * WARPS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t s_mask[WARPS][STAGES];
    const int warp = threadIdx.x >> 5;
    const int32_t rows_per_seq = p.kv_heads * p.n_chunks, ranks = p.cluster, rank = blockIdx.x % ranks;
    const int32_t b = (int32_t)(blockIdx.x / ranks) / rows_per_seq;
    const int32_t head = (int32_t)(blockIdx.x / ranks) - b * rows_per_seq;
    float* const scratch =
        reinterpret_cast<float*>(smem + (size_t)WARPS * STAGES * Loader::STAGE_BYTES) + (size_t)warp * M::SCRATCH;
    sbt_ptx::griddep_wait();
    const AttnRow row = row_of<M::TOK>(p, b);
    const int32_t w = WARPS * ranks, me = rank * WARPS + warp, size = row.tiles / w, more = row.tiles - size * w;
    const int32_t mine = size + (me < more);
    Loader loader(p, smem + (size_t)warp * STAGES * Loader::STAGE_BYTES, s_mask[warp], row, head,
                  me * size + min(me, more), 0, mine);
    M m;
    m.load_q(p, row, head, scratch);
    int stage = 0;
#pragma unroll 1
    for (int32_t i = 0; i < mine; ++i) loader.do_tile(m, stage, scratch);

    // the block's warps, then the cluster's blocks: each block finishes a share of the elements
    float* const s_o = reinterpret_cast<float*>(smem);            // [WARPS][N], then [N] of the block
    float2* const s_ml = reinterpret_cast<float2*>(s_o + (WARPS + 1) * N);
    float* const b_o = s_o + WARPS * N;
    float2* const b_ml = s_ml + WARPS * M::HEADS;
    cp_wait<0>();
    __syncthreads();
    m.put_part(s_o + warp * N, s_ml + warp * M::HEADS);
    __syncthreads();
    for (int i = threadIdx.x; i < N; i += THREADS) {
        float top, l;
        b_o[i] = attn_join<M>(s_o, s_ml, N, M::HEADS, WARPS, i, &top, &l);
        if (i < M::HEADS) b_ml[i] = make_float2(top, l);
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int32_t kvh = head / p.n_chunks, h0 = (head - kvh * p.n_chunks) * p.chunk;
    const int32_t heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
    for (int i = rank * THREADS + threadIdx.x; i < N; i += ranks * THREADS) {
        const int h = i % M::HEADS, d = i / M::HEADS;
        if (h >= heads || d >= p.head_dim) continue;
        float top = -CUDART_INF_F, l = 0.f, x = 0.f;
        for (int r = 0; r < ranks; ++r) {
            const float2 ml = *cluster.map_shared_rank(b_ml + h, r);
            const float o = *cluster.map_shared_rank(b_o + i, r);
            const float t = fmaxf(top, ml.x), ts = t == -CUDART_INF_F ? 0.f : t;
            const float a = exp2_fast(top - ts), c = exp2_fast(ml.x - ts);
            top = t;
            l = l * a + ml.y * c;
            x = x * a + o * c;
        }
        const int32_t qh = kvh * p.group + h0 + h;
        reinterpret_cast<typename M::T*>(p.out)[b * p.ld_out + qh * p.ld_oh + d] = M::from_float(x * inverse(l));
        if (d == 0 && p.lse) p.lse[(int64_t)b * p.q_heads + qh] = log_sum(top, l);
    }
    cluster.sync();  // no block leaves while another reads its shared memory
}

// Joins the parts of the cut rows, each row's in the order of the line.  With
// kJoinDirect descriptors or fewer there is a block for every piece (`direct`
// float4s of the [DP][HEADS] state) of every row; groups of threads go through
// its parts side by side and join in shared memory.  With more, the first blocks,
// one or two per descriptor, give a row of up to kJoinFew parts to their threads,
// a float4 each; rows of more parts are few (their parts are blocks' and add up
// to the grid's), and kJoinExtra blocks per SM look which they are and share
// their pieces out.
// kJoinFew: 64 sequences up to 4096 112 us at 4, 97 at 8 and 16; 8 up to 8192 36 us at 8, 41 at 16.
constexpr int kJoinThreads = 256, kJoinFew = 8, kJoinDirect = 64, kJoinExtra = 2, kJoinMaxDesc = 8192;

template <class M, int WARPS>
__global__ void __launch_bounds__(kJoinThreads) k_attention_join(const AttnParams p, int32_t n_desc, int32_t direct) {
    using namespace sbt_attn;
    constexpr int HEADS = M::HEADS, N = M::HEADS * M::DP, MH = HEADS < 4 ? HEADS : 4;  // MH: different heads in one float4
    __shared__ float s_m[kJoinThreads][MH], s_l[kJoinThreads][MH];
    __shared__ float4 s_o[kJoinThreads];
    __shared__ uint32_t s_many[kJoinMaxDesc / 32];
    sbt_ptx::griddep_wait();

    // parts of the first's block, of the blocks between, of the last's
    struct Count {
        int f, b, n;
    };
    auto count = [](const AttnDesc& e) {
        const int bf = e.first / WARPS, bl = e.last / WARPS;
        Count c;
        c.f = (e.joined & 1) ? 1 : min(e.last, bf * WARPS + WARPS - 1) - e.first + 1;
        c.b = bl > bf ? bl - bf - 1 : 0;
        c.n = c.f + c.b + (bl == bf ? 0 : (e.joined & 2) ? 1 : e.last - bl * WARPS + 1);
        return c;
    };
    auto slot = [](const AttnDesc& e, const Count& c, int i) -> int64_t {
        const int bf = e.first / WARPS;
        if (i < c.f) return (e.joined & 1) ? 2ll * bf * WARPS : 2ll * (e.first + i) + (i == 0 ? e.first_slot : 0);
        i -= c.f;
        return i < c.b ? 2ll * (bf + 1 + i) * WARPS : 2ll * ((int64_t)(e.last / WARPS) * WARPS + i - c.b);
    };
    struct State {
        float m[MH], l[MH], o[4];
        __device__ __forceinline__ State() {
#pragma unroll
            for (int k = 0; k < MH; ++k) m[k] = -CUDART_INF_F, l[k] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = 0.f;
        }
        __device__ __forceinline__ void add(const float* pm, const float* pl, const float4& x) {
            const float px[4] = {x.x, x.y, x.z, x.w};
            float a[MH], b[MH];
#pragma unroll
            for (int k = 0; k < MH; ++k) {
                const float top = fmaxf(m[k], pm[k]), ts = top == -CUDART_INF_F ? 0.f : top;
                a[k] = exp2_fast(m[k] - ts), b[k] = exp2_fast(pm[k] - ts);
                m[k] = top;
                l[k] = l[k] * a[k] + pl[k] * b[k];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = o[k] * a[k % MH] + px[k] * b[k % MH];
        }
    };
    // parts g, g + step, .. of the float4 that starts at element `at`
    auto gather = [&](const AttnDesc& e, const Count& c, int at, int g, int step) {
        State s;
        const int head = at % HEADS;
#pragma unroll 4
        for (int i = g; i < c.n; i += step) {
            const int64_t q = slot(e, c, i);
            float pm[MH], pl[MH];
#pragma unroll
            for (int k = 0; k < MH; ++k) {
                const float2 ml = p.part_ml[q * HEADS + head + k];
                pm[k] = ml.x, pl[k] = ml.y;
            }
            s.add(pm, pl, *reinterpret_cast<const float4*>(p.part_o + q * N + at));
        }
        return s;
    };
    auto write = [&](const AttnDesc& e, const State& s, int at) {
        const int32_t h0 = e.chunk * p.chunk, heads = p.group - h0 < p.chunk ? p.group - h0 : p.chunk;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = (at + k) % HEADS, d = (at + k) / HEADS;
            if (h >= heads || d >= p.head_dim) continue;
            const int32_t qh = e.kvh * p.group + h0 + h;
            reinterpret_cast<typename M::T*>(p.out)[e.b * p.ld_out + qh * p.ld_oh + d] =
                M::from_float(s.o[k] * inverse(s.l[k % MH]));
            if (d == 0 && p.lse) p.lse[(int64_t)e.b * p.q_heads + qh] = log_sum(s.m[k % MH], s.l[k % MH]);
        }
    };

    constexpr int PER_ROW = (N + 4 * kJoinThreads - 1) / (4 * kJoinThreads);
    const int first = direct ? 0 : n_desc * PER_ROW;
    if ((int32_t)blockIdx.x < first) {
        const AttnDesc e = p.desc[blockIdx.x / PER_ROW];
        if (!e.valid) return;
        const Count c = count(e);
        const int at = ((blockIdx.x % PER_ROW) * kJoinThreads + threadIdx.x) * 4;
        if (c.n <= kJoinFew && at < N) write(e, gather(e, c, at, 0, 1), at);
        return;
    }
    // piece number i of a row of many parts
    auto do_piece = [&](const AttnDesc& e, const Count& c, int piece, int i) {
        const int t = threadIdx.x & (piece - 1), g = threadIdx.x / piece, groups = kJoinThreads / piece;
        const int at = (i * piece + t) * 4;
        State s;
        if (at < N) s = gather(e, c, at, g, groups);
#pragma unroll
        for (int k = 0; k < MH; ++k) s_m[threadIdx.x][k] = s.m[k], s_l[threadIdx.x][k] = s.l[k];
        s_o[threadIdx.x] = make_float4(s.o[0], s.o[1], s.o[2], s.o[3]);
        __syncthreads();
        if (g == 0 && at < N) {
            for (int w = 1; w < groups && w < c.n; ++w)
                s.add(s_m[w * piece + t], s_l[w * piece + t], s_o[w * piece + t]);
            write(e, s, at);
        }
        __syncthreads();
    };
    if (direct) {
        const int pieces = (N / 4 + direct - 1) / direct, item = blockIdx.x - first;
        const AttnDesc e = p.desc[item / pieces];
        if (!e.valid) return;
        do_piece(e, count(e), direct, item % pieces);
        return;
    }
    // which descriptors have many parts, the same list in every block
    int rows = 0;
    for (int d0 = 0; d0 < n_desc; d0 += kJoinThreads) {
        const int d = d0 + threadIdx.x;
        bool many = false;
        if (d < n_desc) {
            const AttnDesc e = p.desc[d];
            many = e.valid && count(e).n > kJoinFew;
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, many);
        if ((threadIdx.x & 31) == 0 && d < n_desc) s_many[d >> 5] = bits;
        rows += __syncthreads_count(many);
    }
    const int blocks = gridDim.x - first;
    const int piece = rows * (N / 64) <= blocks ? 16 : 64, pieces = (N / 4 + piece - 1) / piece;
    int item = blockIdx.x - first, base = 0;    // of the pieces of all listed rows; first one of the row at hand
    for (int w = 0; w * 32 < n_desc && base < rows * pieces; ++w)
        for (uint32_t bits = s_many[w]; bits; bits &= bits - 1, base += pieces)
            for (; item < base + pieces; item += blocks) {
                const AttnDesc e = p.desc[w * 32 + __ffs(bits) - 1];
                do_piece(e, count(e), piece, item - base);
            }
}

// Enqueues the kernel and the join, or the cluster form, for one instantiation.
template <class M, int STAGES, int WARPS, int BLOCKS>
sbt_status sbt_attention_enqueue(sbt_context* ctx, AttnParams p, cudaStream_t stream) {
    constexpr size_t ring = (size_t)WARPS * (STAGES * 2 * M::TOK * M::PITCH + M::SCRATCH * sizeof(float));
    constexpr size_t states = (size_t)(WARPS + 1) * M::HEADS * (M::DP * sizeof(float) + sizeof(float2));
    constexpr size_t smem = ring > states ? ring : states;
    p.tile_in_page = p.page_size.d % M::TOK == 0;
    const int resident = sbt_resident_blocks<k_paged_attention<M, STAGES, WARPS, BLOCKS>>(ctx, 32 * WARPS, smem);
    const int64_t rows = (int64_t)p.batch * p.kv_heads * p.n_chunks;
    // The longest row there can be, in tiles.
    const int64_t longest = sbt_cdiv(p.window > 0 && p.window < p.max_len ? (int64_t)p.window + M::TOK : p.max_len, M::TOK);
    // A cluster per row where all clusters fit at once and a warp gets kClusterTiles tiles at most: below
    // that the second launch and the way through memory cost more than uneven work.  bf16, 32 and 8 heads
    // of 128: one sequence of 512 7.3 us and 11.5 without, of 4096 11.0 and 12.8; 16 of 2048 26.7 and 32.4.
    int ranks = (int)(resident / rows < kClusterMost ? resident / rows : kClusterMost);
    if (ranks > sbt_cdiv(longest, WARPS)) ranks = (int)sbt_cdiv(longest, WARPS);
    if (ranks < 1) ranks = 1;
    if (rows * ranks <= resident && longest <= (int64_t)ranks * WARPS * kClusterTiles) {
        p.cluster = ranks;
        sbt_resident_blocks<k_paged_attention_cluster<M, STAGES, WARPS, BLOCKS>>(ctx, 32 * WARPS, smem);
        if (sbt_status st = sbt_cuda_check(
                sbt_launch_dependent_cluster(k_paged_attention_cluster<M, STAGES, WARPS, BLOCKS>,
                                             dim3((unsigned)(rows * ranks)), dim3(32 * WARPS), (unsigned)ranks, smem,
                                             stream, p),
                "paged_attention launch"))
            return st;
        return sbt_after_launch(ctx, "paged_attention");
    }
    int grid = std::min(resident, ctx->sm_count * kAttnMaxWarps / WARPS);
    grid = std::min(grid, kJoinMaxDesc / WARPS);
    p.desc_by_row = rows <= (int64_t)grid * WARPS;
    sbt_status st = sbt_cuda_check(sbt_launch_dependent(k_paged_attention<M, STAGES, WARPS, BLOCKS>, dim3(grid),
                                                        dim3(32 * WARPS), smem, stream, p),
                                   "paged_attention launch");
    if (st || (st = sbt_after_launch(ctx, "paged_attention"))) return st;
    const int n_desc = p.desc_by_row ? (int)rows : grid * WARPS;
    const int quads = M::HEADS * M::DP / 4;
    int direct = 0, blocks = n_desc * (int)sbt_cdiv(quads, kJoinThreads) + kJoinExtra * ctx->sm_count;
    if (n_desc <= kJoinDirect) {
        // the smallest pieces of which two blocks per SM are enough: 8 sequences up to 8192 34.2 us; 35.8 with
        // fixed pieces for long rows and a thread per float4 for rows of up to kJoinFew parts
        direct = 8;
        while (direct < 64 && n_desc * sbt_cdiv(quads, direct) > 2 * ctx->sm_count) direct *= 2;
        blocks = n_desc * (int)sbt_cdiv(quads, direct);
    }
    if ((st = sbt_cuda_check(sbt_launch_dependent(k_attention_join<M, WARPS>, dim3(blocks),
                                                  dim3(kJoinThreads), 0, stream, p, n_desc, direct),
                             "paged_attention join launch")))
        return st;
    return sbt_after_launch(ctx, "paged_attention join");
}

sbt_status sbt_attention_f32(sbt_context* ctx, const AttnParams& p, cudaStream_t stream);
