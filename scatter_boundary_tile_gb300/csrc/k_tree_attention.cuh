// Attention of several new tokens per sequence over a paged key-value cache: a
// prompt's next piece or a tree of drafted tokens.
//
// For a query row (a token's query head) with scores s_t = scale q . k_t over
// the positions it sees, one pass over the cache keeps a reference m, the sum
// l = sum 2^(s'_t - m) and the vector o = sum 2^(s'_t - m) v_t (s' = s log2 e).
// m is the largest score seen when it was last taken; it is taken again, and l
// and o rescaled, only when a score passes it by SLACK (2^8; fp16 2^6), so a
// 2^(s' - m) is at most that and o rarely has to be touched outside the matrix
// unit.  Two such states over disjoint positions join by the rule of the softmax.
//
// The rows of one sequence and key-value head, n tokens times `group` query
// heads, go through tcgen05 in tiles of 128: S = Q K^T and O += P V with K and V
// tiles of 64 positions in shared memory (rows of 128 bytes, swizzled: K read
// K-major, V MN-major), S, P and O in TMEM; S is double, so that tile k + 1 is
// multiplied while tile k is in the softmax.  MT = 1: 128 rows, two blocks an SM
// (the one's softmax runs under the other's products).  MT = 2: planes of 256
// rows that share each tile of K and V; where a plane has 128 rows or fewer the
// instructions of the other half are left out.  Entries of more rows have more
// planes, each a line of its own.
//
// P is the sum of two 16-bit numbers (16 significant bits with bf16, 22 with fp16),
// as in the attention of single tokens: one would add to the output's error as much
// as the output's own rounding.  Where planes of 256 rows are full the second costs
// 12 to 25 % (48 sequences of 64/8 heads, fp16: trees of 1 to 64 tokens 324 and 364 us
// with one and two, 32 tokens 362 and 436, 64 tokens 705 and 880), elsewhere nothing.
// fp16 ones are 2^SHIFT p, so that small ones are not lost among the subnormals.
//
// Roles.  A warp for every 32 rows does the softmax, a row a thread: it also
// reads the row's query into shared memory and writes the row's output.  Two warps
// copy K and V by the tensor copy engine, where pages hold whole boxes and strides
// are multiples of 16 bytes; otherwise three warps do with cp.async, from any
// stride and page size.  A warp for every 128 rows issues the products: all
// of its lanes walk and wait, one issues (an instruction takes ~30 cycles to
// issue so, 74 from a branch that one lane takes).
//
// Split.  All (entry, key-value head, plane) lines, cut into tiles, lie on one
// line on which every block gets an even range; lengths are read on the device.
// (Planes in turn on one range: 463 us for the batch below instead of 369, one number
// per probability.)
// Rows wholly inside a range are written by their block; of a line cut by range
// borders each block writes its state to the workspace and k_tree_join adds them
// in the order of the line.
//
// A masked position's score is replaced before the softmax, its P is zero.  Its
// V would still meet that zero: among the new tokens, which one row sees and
// another does not, the softmax warps take infinities and NaN out of the tile,
// and put them, after the last tile, on the rows that do see them.
//
// Measured (GB300, 128 elements a head; the cache at the copy rate in brackets).
// MT = 1: one sequence, 32 tokens on 16384 positions, 32/8 heads, bf16 38 us (10),
// on 131072 114 (79), on 2048 25: the launches, a cold instruction cache and the
// join are most of a short call.  MT = 2: 48 sequences, 32 tokens on 8192
// positions, 64/8 heads, fp16 450 us (246); trees of 1 to 64 tokens on contexts to
// 8191 385 (130).  There a tile takes ~1900 cycles, the round of the warp that issues
// the products: P seen 270, product issued 540, next scores 860, beside the other
// half's.  The softmax, 1180 cycles from scores to P, waits for it (one number per
// probability: 1650 cycles, and it waits for the softmax).  The products alone are
// ~1540 by their sizes (with 64 columns they read Q from shared memory at 3/2 of the
// time that their multiplication takes).
//
// Every wait is bounded; one that runs out sets the device status word, and the
// kernel drains and returns.
#pragma once

#include "k_paged_attention.cuh"
#include "sbt_num.cuh"

namespace sbt_tree {

using namespace sbt_ptx;
using namespace sbt_num;
using sbt_attn::Line;

constexpr int kTok = 64, kRows = 128, kLoaders = 96;
constexpr int kLineCost = 3;      // what starting and ending a line costs, in tiles
constexpr int kBits = 16;         // tiles whose visible positions are remembered
constexpr int kJoin = 256;

struct TreeDesc {
    int32_t valid, b, h, plane, first, last, first_slot, pad;
};

struct TreeAttnParams {
    const char *q, *k, *v;
    char* out;
    float* lse;
    const int32_t *cu, *table, *lens, *seq;
    const uint32_t* mask;
    int64_t ld_q, ld_qh, ld_out, ld_oh;        // elements
    int64_t ld_page, ld_slot, ld_head;         // elements
    int64_t ld_table, n_pages, ld_mask;
    int32_t rows, batch, max_new, q_heads, kv_heads, n_seq, head_dim, max_len;
    int32_t planes;                            // MT * 128 rows each that an entry may need
    int32_t copy_kv, q_vec, out_vec;           // bytes of a copy by lanes; q and out as 16-byte vectors
    int32_t desc_by_line;                      // descriptors by line (there are no more lines than blocks), else by block
    sbt_fastdiv group, page_size;
    float scale;                               // |scale| log2 e, not zero
    int32_t negate;                            // the scale is negative
    unsigned int* status;
    uint64_t wait_ns;
    int32_t withhold;                          // test hook: no block signals its first tile
    TreeDesc* desc;
    float2* part_ml;                           // [2 blocks][MT * 128]
    float4* part_o;                            // [2 blocks][DP / 4][MT * 128]
};

// Keys and values as tensors of pages, heads, slots and elements.
struct TreeMaps {
    CUtensorMap k, v;
    bool use;
};

// Entry b (its tokens are the rows q0 .. q0 + n - 1 of q, the last n of len positions; n = 0: none, or left out) and
// one plane of its rows.
struct TreeRow {
    int32_t b, q0, n, len, seq;
    int32_t plane, count, tiles;               // query rows, and tiles they see
};

__device__ __forceinline__ void set_plane(const TreeAttnParams& p, TreeRow& r, int32_t plane, int32_t R) {
    const int64_t all = r.n * (int64_t)p.group.d, first = (int64_t)plane * R;
    r.plane = plane;
    r.count = (int32_t)max((int64_t)0, min((int64_t)R, all - first));
    r.tiles = 0;
    if (r.count == 0 || r.seq < 0) return;
    // without a mask no row of the plane sees past its last token
    const int32_t last = (int32_t)sbt_div(p.group, (uint32_t)(first + r.count - 1));
    const int32_t hi = p.mask ? r.len : r.len - r.n + last + 1;
    r.tiles = hi > 0 ? (hi + kTok - 1) / kTok : 0;
}

__device__ __forceinline__ TreeRow row_of(const TreeAttnParams& p, int32_t b, int32_t R) {
    TreeRow r = {b, 0, 0, 0, -1, 0, 0, 0};
    const int32_t c0 = sbt_ld(p.cu + b), c1 = sbt_ld(p.cu + b + 1), s = p.seq ? sbt_ld(p.seq + b) : b;
    const bool held = s >= 0 && s < p.n_seq;
    const int32_t len = held ? sbt_ld(p.lens + s) : 0;         // on its way beside cu
    const int64_t n = (int64_t)c1 - c0;
    if (c0 < 0 || c1 > p.rows || n <= 0 || n > p.max_new) return r;
    r.q0 = c0, r.n = (int32_t)n;
    if (held) r.seq = s, r.len = min(max(len, 0), p.max_len);
    set_plane(p, r, 0, R);
    return r;
}

// Planes that an entry's rows fill.
__device__ __forceinline__ int32_t planes_of(const TreeAttnParams& p, const TreeRow& r, int32_t R) {
    return (int32_t)((r.n * (int64_t)p.group.d + R - 1) / R);
}

// Places of one head's lines, a line for every plane that sees anything.
__device__ __forceinline__ int64_t head_places(const TreeAttnParams& p, TreeRow r, int32_t R) {
    int64_t sum = 0;
    for (int32_t i = 0; i < planes_of(p, r, R); ++i) {
        set_plane(p, r, i, R);
        if (r.tiles) sum += r.tiles + kLineCost;
    }
    return sum;
}

// The lines of a range, one after another; every role walks it by itself.
struct Walk {
    const TreeAttnParams& p;
    int32_t R;
    TreeRow row;
    int32_t h, t;          // key-value head; first tile of the segment
    int64_t u, end;        // its place; the range's end

    // The tiles of the segment at hand.
    __device__ __forceinline__ int32_t tiles() const { return (int32_t)min((int64_t)(row.tiles - t), end - u); }
    // The first line from here on (plane, head, entry) that sees anything.
    __device__ __forceinline__ void find() {
        while (true) {
            for (const int32_t n = planes_of(p, row, R); row.plane < n; set_plane(p, row, row.plane + 1, R))
                if (row.tiles) return;
            if (row.seq >= 0 && row.n && ++h < p.kv_heads) {
                set_plane(p, row, 0, R);
                continue;
            }
            h = 0;
            if (row.b + 1 >= p.batch) return;
            row = row_of(p, row.b + 1, R);
        }
    }
    __device__ __forceinline__ void next(int32_t done) {
        u += done;
        t += done;
        if (t < row.tiles) return;
        u += kLineCost;
        t = 0;
        if (u >= end) return;
        set_plane(p, row, row.plane + 1, R);
        find();
    }
};

// D (+)= A B, A in shared memory (`a` the low half of its descriptor) or, _ts, in TMEM (`a` its address); the high
// halves of the descriptors are the same for all tiles.  The issuing thread has a few instructions for each of these,
// so the operands come as sums of a word that the warp shares and a constant.
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "n"(ACC)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 lanes x 8 (or 32) consecutive 32-bit columns, from thread i of the warp to lane (base lane + i).
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// The largest of three; NaN counts for nothing.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int KIND>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (KIND == kBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <int KIND>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (KIND == kBF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Infinity or NaN.
template <int KIND>
__device__ __forceinline__ bool special(uint16_t x) {
    constexpr uint16_t e = KIND == kBF16 ? 0x7F80 : 0x7C00;
    return (x & e) == e;
}

template <int KIND, int DP, int MT, bool TMA>
struct TreeShape {
    static constexpr int WARPS = 4 * MT + (TMA ? 2 : kLoaders / 32) + MT, THREADS = 32 * WARPS;
    // (registers are bounded for whole warps on each of the SM's four partitions)
    static constexpr int BLOCKS = MT == 1 && DP <= 128 ? 2 : 1;
    static constexpr int R = MT * kRows;
    static constexpr uint32_t Q_TILE = kRows * DP * 2, SLOT = kTok * DP * 2;
    static constexpr uint32_t MOST = (BLOCKS == 2 ? 113 : 227) * 1024 - 8192 - 1536 - MT * Q_TILE;
    static constexpr int SLOTS = MOST / SLOT < 8 ? MOST / SLOT : 8;
    static constexpr size_t SMEM = 1024 + 512 + MT * Q_TILE + SLOTS * SLOT;
    static constexpr uint32_t O_COL = MT * 2 * kTok;            // S (and P): [MT][2][64], then O: [MT][DP]
    static constexpr uint32_t COLS = O_COL + MT * DP <= 256 ? 256 : 512;
    static constexpr int BARS = 2 * SLOTS + 8 * MT;
    static constexpr float SLACK = KIND == kF16 ? 6.f : 8.f;    // see the head of the file
    static constexpr float SHIFT = KIND == kF16 ? 9.f : 0.f;
    static_assert(SLOTS >= 4, "K two tiles ahead of V, and two more on their way");
    static_assert(BARS * 8 + kBits * 8 + 16 <= 512, "barriers and notes fit their place");
};

enum : unsigned int { kCodeTreeLoad = 0x10000, kCodeTreeMma = 0x20000, kCodeTreeSoft = 0x40000 };

template <int KIND, int DP, int MT, bool TMA>
__global__ void __launch_bounds__((TreeShape<KIND, DP, MT, TMA>::WARPS + 3) / 4 * 128, TreeShape<KIND, DP, MT, TMA>::BLOCKS)
    k_tree_attention(const TreeAttnParams p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
    typedef TreeShape<KIND, DP, MT, TMA> S;
    constexpr int WARPS = S::WARPS, THREADS = S::THREADS, R = S::R, NS = S::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t s_warp[WARPS];
    __shared__ int64_t s_first[THREADS];
    __shared__ TreeRow s_row;
    __shared__ int64_t s_offsets[TMA ? 1 : kLoaders / 32][2 * kTok];
    __shared__ volatile int s_uses[NS];  // copies by the engine that each slot has taken
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* const q_s = smem;
    uint8_t* const ring = smem + MT * S::Q_TILE;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(ring + NS * S::SLOT);
    uint64_t* const s_bits = bars + S::BARS;                              // [kBits] positions of a tile that are on a page
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(s_bits + kBits);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* const s_special = abort_flag + 1;                       // a V among the new positions held infinity or NaN
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (NS + s); };
    auto q_full = [&](int m) { return bar0 + 8u * (2 * NS + 8 * m); };
    auto all_done = [&](int m) { return q_full(m) + 8u; };
    auto s_full = [&](int m, int buf) { return q_full(m) + 8u * (2 + buf); };
    auto p_ready = [&](int m, int buf) { return q_full(m) + 8u * (4 + buf); };
    // one for each of two tiles: a wait for tile k comes after tile k - 2 is done and before k + 2 can be, so that
    // the parity names the phase
    auto pv_done = [&](int m, int buf) { return q_full(m) + 8u * (6 + buf); };
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) mbar_init(full(s), TMA ? 1 : kLoaders), mbar_init(empty(s), MT);
        for (int m = 0; m < MT; ++m) {
            mbar_init(q_full(m), kRows), mbar_init(all_done(m), 1);
            for (int b = 0; b < 2; ++b) mbar_init(s_full(m, b), 1), mbar_init(p_ready(m, b), kRows), mbar_init(pv_done(m, b), 1);
        }
        for (int i = 0; i < NS; ++i) s_uses[i] = 0;
        *abort_flag = 0;
        *s_special = 0;
        fence_mbar_init();
    }
    if (warp == WARPS - 1) {
        tmem_alloc(smem_u32(tmem_slot), S::COLS);
        tmem_relinquish();
    }
    if (!TMA && p.head_dim < DP) {  // columns past the head size stay zero for the whole call
        uint4* const w = reinterpret_cast<uint4*>(smem);
        for (uint32_t i = threadIdx.x; i < (MT * S::Q_TILE + NS * S::SLOT) / 16; i += THREADS) w[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    // ---- the line, and this block's range of it
    const int32_t c = blockIdx.x;
    auto places = [&](int32_t b, TreeRow& r) { return head_places(p, r = row_of(p, b, R), R) * p.kv_heads; };
    const bool one_step = p.batch <= THREADS;  // every thread holds its own entry's places
    int64_t total = 0, at = 0, mine_places = 0;
    TreeRow my_row;
    if (one_step) {
        if ((int32_t)threadIdx.x < p.batch) mine_places = places(threadIdx.x, my_row);
        at = sbt_attn::block_scan<WARPS>(mine_places, &total, s_warp);
    } else {
        for (uint32_t b = threadIdx.x; b < (uint32_t)p.batch; b += THREADS) total += places((int32_t)b, my_row);
        int64_t sum;
        sbt_attn::block_scan<WARPS>(total, &sum, s_warp);
        total = sum;
    }
    const int64_t G = min(total, (int64_t)gridDim.x);
    bool idle = c >= G;
    const Line line(total, G > 0 ? G : 1);
    const int64_t u0 = idle ? total : line.start(c), u1 = idle ? total : line.start(c + 1);
    int32_t b_first = 0;
    int64_t u_first = 0;
    {
        int64_t before = 0;
        for (uint32_t b0 = 0; b0 < (uint32_t)p.batch && before <= u0; b0 += THREADS) {
            int64_t sum = total;
            if (!one_step) {
                const uint32_t b = b0 + threadIdx.x;
                at = before + sbt_attn::block_scan<WARPS>(b < (uint32_t)p.batch ? places((int32_t)b, my_row) : 0, &sum, s_warp);
            }
            s_first[threadIdx.x] = at;
            __syncthreads();
            if (before <= u0 && u0 < before + sum) {
                for (int i = lane; i < THREADS; i += 32) {
                    const int64_t e = i + 1 < THREADS ? s_first[i + 1] : before + sum;
                    const uint32_t hit = __ballot_sync(0xffffffffu, s_first[i] <= u0 && u0 < e);
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
    if (!p.desc_by_line && threadIdx.x == 0) p.desc[blockIdx.x].valid = 0;

    if (one_step && !idle && (int32_t)threadIdx.x == b_first) s_row = my_row;
    __syncthreads();
    Walk start = {p, R, {}, 0, 0, 0, u1};
    if (!idle) {
        start.row = one_step ? s_row : row_of(p, b_first, R);
        set_plane(p, start.row, 0, R);
        const int64_t width = head_places(p, start.row, R);
        start.h = (int32_t)sbt_attn::divide(u0 - u_first, width);
        int64_t line_u = u_first + start.h * width;              // of the line that holds u0
        while (start.row.tiles == 0 || u0 >= line_u + start.row.tiles + kLineCost) {
            if (start.row.tiles) line_u += start.row.tiles + kLineCost;
            set_plane(p, start.row, start.row.plane + 1, R);
        }
        line_u += kLineCost;
        start.u = u0 > line_u ? u0 : line_u;
        start.t = (int32_t)(start.u - line_u);
        idle = start.u >= u1;  // nothing but a line's empty places
    }

    if (idle) {
    } else if (TMA && (warp == 4 * MT || warp == 4 * MT + 1)) {
        // ------------------------------------------------------------ copies by the tensor copy engine
        // One warp copies K and one V: to start a tile's copies takes a warp ~900 cycles (one for both took longer than
        // the products: 8 trees of 48 tokens on 8192 positions, 32/8 heads of 128, 92 us, and 82 so; but 48 of 32 tokens,
        // 64/8 heads in fp16, 383 and 393; both with one number per probability).
        // A tile is a box of 64 elements and a page's positions (64 at most) for every 128 bytes of its rows; a lane
        // starts one of them.  A page that is not there is a coordinate outside the tensor, which reads as zeros.
        const bool is_v = warp != 4 * MT;
        const CUtensorMap* const map = is_v ? &v_map : &k_map;
        const int per_page = min((int)p.page_size.d, kTok), boxes = kTok / per_page * (DP / 64);
        const int mine = lane / (DP / 64), x = lane % (DP / 64) * 64;  // page of the tile, first element
        const uint32_t box_at = smem_u32(ring) + (x / 64) * kTok * 128 + mine * per_page * 128;
        int slot = 0, tile_no = 0;
        uint32_t phase = 1;  // the first pass finds the slots empty
        bool ok = true;
        for (Walk w = start; ok && w.u < w.end;) {
            const TreeRow& row = w.row;
            const int32_t T = w.tiles();
            // pages are asked for four tiles ahead: of four tiles, by their numbers modulo 4
            int32_t page[4], at[4];
            auto look_up = [&](int32_t it, int32_t& page, int32_t& at) {
                const int32_t pos = (w.t + it) * kTok + mine * per_page;
                page = -1, at = 0;
                if (lane < boxes && it < T && pos < row.len) {
                    const uint32_t j = sbt_div(p.page_size, (uint32_t)pos);
                    at = pos - (int32_t)(j * p.page_size.d);
                    page = sbt_ld(p.table + (int64_t)row.seq * p.ld_table + j);
                }
            };
            auto skip = [&](int slots) {  // three at most, less than there are
                slot += slots;
                if (slot >= NS) slot -= NS, phase ^= 1;
            };
            auto tile = [&](int32_t page, int32_t at) {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty(slot), phase, p.wait_ns, abort_flag, p.status, kCodeTreeLoad))) {
                    ok = false;
                    return;
                }
                // the test hook's first tile is neither announced nor started
                const bool withheld = p.withhold && !is_v && tile_no == 0;
                if (lane == 0 && !withheld) {
                    s_uses[slot] = s_uses[slot] + 1;
                    mbar_arrive_expect_tx(full(slot), S::SLOT);
                }
                __syncwarp();
                if (lane < boxes && !withheld)
                    tma_load_4d(box_at + slot * S::SLOT, map, x, at, w.h, page >= 0 && page < p.n_pages ? page : -1, full(slot));
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) look_up(i, page[i], at[i]);
            // the slots go to K K V K V .. K V V: K runs two tiles ahead of V, as the products do
            if (is_v) skip(T > 1 ? 2 : 1);
            for (int32_t it0 = 0; ok && it0 < T; it0 += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int32_t it = it0 + i;
                    if (ok && it < T) {
                        if (!is_v) {
                            uint64_t bits = 0;
                            if (lane < boxes && x == 0 && page[i] >= 0 && page[i] < p.n_pages)
                                bits = (per_page == kTok ? ~0ull : (1ull << per_page) - 1) << (mine * per_page);
                            const uint32_t lo = __reduce_or_sync(0xffffffffu, (uint32_t)bits);
                            const uint32_t hi = __reduce_or_sync(0xffffffffu, (uint32_t)(bits >> 32));
                            if (lane == 0) s_bits[tile_no & (kBits - 1)] = lo | (uint64_t)hi << 32;
                            __syncwarp();
                        }
                        tile(page[i], at[i]);
                        ++tile_no;
                        look_up(it + 4, page[i], at[i]);
                        const bool last = it + 1 == T;
                        if (is_v)
                            skip(it + 2 >= T ? 1 : 2);
                        else
                            skip(last ? (T == 1 ? 2 : 3) : it == 0 ? 1 : 2);
                    }
                }
            w.next(T);
        }
    } else if (!TMA && warp >= 4 * MT && warp < WARPS - MT) {
        // ------------------------------------------------------------ copies by lanes
        const int tid = threadIdx.x - 4 * MT * 32;
        int item = 0, landed = 0;          // tiles begun, and signalled as landed
        bool ok = true;
        int tile_no = 0;
        const uint32_t ring_u32 = smem_u32(ring);
        constexpr int LPR = DP <= 64 ? 8 : DP <= 128 ? 16 : 32, RPI = 32 / LPR;  // lanes of a row, 16 bytes each; rows at a time
        const int lw = tid >> 5, byte0 = (lane % LPR) * 16, r0 = lane / LPR, row_bytes = p.head_dim * 2;
        int64_t* const s_off = s_offsets[lw];  // of the rows of two tiles: byte offsets, -1 where there is none
        // place of a byte of row r
        auto place = [](uint32_t base, int r, int byte) {
            return base + (uint32_t)(byte >> 7) * kTok * 128u + r * 128u + ((((byte >> 4) & 7) ^ (r & 7)) << 4) + (byte & 15);
        };
        // This lane's rows of a tile are row0, row0 + STEP, ..; their places, less the rows' pitch, repeat.
        constexpr int STEP = RPI * (kLoaders / 32), N = (kTok + STEP - 1) / STEP;
        constexpr int PERIOD = STEP % 8 == 4 ? 2 : STEP % 4 == 2 ? 4 : 8;
        const int row0 = lw * RPI + r0;
        uint32_t at_place[PERIOD];
#pragma unroll
        for (int i = 0; i < PERIOD; ++i) at_place[i] = place(0, row0 + i * STEP, byte0) - i * STEP * 128;
        // A whole tile in 16-byte pieces, every row of which is on a page: as few instructions as a copy can take, since
        // three warps start all copies of an SM.
        auto copy_tile = [&](uint32_t dst, const char* src, const int64_t* o) {
            constexpr int BATCH = 6;
            src += byte0;
            if (byte0 < row_bytes)
#pragma unroll
                for (int i0 = 0; i0 < N; i0 += BATCH) {
                    const char* a[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        if (i0 + i < N) a[i] = src + o[min(row0 + (i0 + i) * STEP, kTok - 1)];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        if (i0 + i < N && ((i0 + i + 1) * STEP <= kTok || row0 + (i0 + i) * STEP < kTok))
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + at_place[(i0 + i) % PERIOD] +
                                                                                           (i0 + i) * STEP * 128),
                                         "l"(a[i])
                                         : "memory");
                }
        };
        auto wait_landed = [&](int in_flight) {  // at most so many of this thread's tiles are still on their way
            switch (in_flight) {
                case 0: sbt_attn::cp_wait<0>(); break;
                case 1: sbt_attn::cp_wait<1>(); break;
                case 2: sbt_attn::cp_wait<2>(); break;
                case 3: sbt_attn::cp_wait<3>(); break;
                case 4: sbt_attn::cp_wait<4>(); break;
                case 5: sbt_attn::cp_wait<5>(); break;
                case 6: sbt_attn::cp_wait<6>(); break;
                default: sbt_attn::cp_wait<7>(); break;
            }
        };
        // The same with rows that are not there (zeros) or pieces of less than 16 bytes.
        auto copy_rows = [&](uint32_t dst, uint8_t* dst_p, const char* src, const int64_t* o) {
            const int bytes = p.copy_kv;
            auto at = [&](int r) { return o[r] < 0 ? nullptr : src + o[r]; };
            if (bytes == 16) {
                if (byte0 < row_bytes)
                    for (int r = row0; r < kTok; r += STEP) {
                        const char* const a = at(r);
                        sbt_attn::cp_async16(place(dst, r, byte0), a ? a + byte0 : p.q, a ? 16 : 0);
                    }
            } else {
                for (int r = lw; r < kTok; r += kLoaders / 32) {
                    const char* const a = at(r);
                    for (int byte = lane * bytes; byte < row_bytes; byte += 32 * bytes) {
                        if (bytes == 8)
                            sbt_attn::cp_async8(place(dst, r, byte), a ? a + byte : p.q, a ? 8 : 0);
                        else if (bytes == 4)
                            sbt_attn::cp_async4(place(dst, r, byte), a ? a + byte : p.q, a ? 4 : 0);
                        else
                            *reinterpret_cast<uint16_t*>(dst_p + (place(0, r, byte))) =
                                a ? sbt_ld(reinterpret_cast<const uint16_t*>(a + byte)) : (uint16_t)0;
                    }
                }
            }
        };
        // The oldest tile on its way has landed: it is signalled.
        auto signal = [&]() {
            wait_landed(item - landed - 1);
            const int s = landed % NS;
            fence_proxy_async_smem();
            if (!(p.withhold && landed == 0)) mbar_arrive(full(s));
            ++landed;
        };
        // A free slot for the next tile; tiles that land meanwhile are signalled.
        auto slot_of = [&]() {
            const int s = item % NS, use = item / NS;
            while (use > 0) {
                const bool free = mbar_test_wait(empty(s), (use - 1) & 1);  // must not sleep: tiles may wait to be signalled
                if (__all_sync(0xffffffffu, free)) break;
                if (landed < item) {
                    signal();
                } else if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty(s), (use - 1) & 1, p.wait_ns, abort_flag,
                                                                      p.status, kCodeTreeLoad))) {
                    ok = false;
                    break;
                }
            }
            return s;
        };

        for (Walk w = start; ok && w.u < w.end;) {
            const TreeRow& row = w.row;
            const int32_t T = w.tiles();
            // this lane's two positions of a tile and their pages, -1 where there is none
            int32_t at[2], page[2];
            auto look_up = [&](int32_t it) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int32_t pos = (w.t + it) * kTok + j * 32 + lane;
                    page[j] = -1;
                    if (it < T && pos < row.len) {
                        const uint32_t pg = sbt_div(p.page_size, (uint32_t)pos);
                        at[j] = pos - (int32_t)(pg * p.page_size.d);
                        page[j] = sbt_ld(p.table + (int64_t)row.seq * p.ld_table + pg);  // read when the tile is begun
                    }
                }
            };
            bool all[2] = {false, false};  // of two tiles: every row is on a page
            // tile it of K or V
            auto tile = [&](const char* src, int32_t it) {
                const int s = slot_of();
                if (!ok) return;
                const int64_t* const o = s_off + (it & 1) * kTok;
                if (all[it & 1] && p.copy_kv == 16)
                    copy_tile(ring_u32 + s * S::SLOT, src, o);
                else
                    copy_rows(ring_u32 + s * S::SLOT, ring + s * S::SLOT, src, o);
                sbt_attn::cp_commit();
                ++item;
            };
            auto k_tile = [&](int32_t it) {  // the positions looked up last are this tile's
                bool ok[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    ok[j] = page[j] >= 0 && page[j] < p.n_pages;
                    s_off[(it & 1) * kTok + j * 32 + lane] =
                        ok[j] ? (page[j] * p.ld_page + at[j] * p.ld_slot + w.h * p.ld_head) * 2 : -1;
                }
                const uint32_t lo = __ballot_sync(0xffffffffu, ok[0]), hi = __ballot_sync(0xffffffffu, ok[1]);
                if (tid == 0) s_bits[tile_no & (kBits - 1)] = lo | (uint64_t)hi << 32;
                all[it & 1] = (lo & hi) == ~0u;
                ++tile_no;
                __syncwarp();
                look_up(it + 1);
                tile(p.k, it);
            };
            look_up(0);
            // K runs two tiles ahead of V, as the products do
            k_tile(0);
            if (ok && T > 1) k_tile(1);
            for (int32_t it = 0; ok && it < T; ++it) {
                tile(p.v, it);
                __syncwarp();  // its offsets make room for those of two tiles on
                if (ok && it + 2 < T) k_tile(it + 2);
            }
            w.next(T);
        }
        while (ok && landed < item) signal();
        sbt_attn::cp_wait<0>();
    } else if (warp >= WARPS - MT) {
        // ------------------------------------------------------------ matrix instructions: a warp for each 128 rows
        const int m = warp - (WARPS - MT);
        // The whole warp walks and waits, so that what the instructions take is the same for all lanes; one lane issues.
        auto elected = []() {
            uint32_t yes;
            asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
            return yes != 0;
        };
        const uint32_t type = KIND == kBF16 ? (1u << 7) | (1u << 10) : 0u;
        const uint32_t idesc_s = (1u << 4) | type | ((kTok >> 3) << 17) | ((kRows >> 4) << 24);
        const uint32_t idesc_o = (1u << 4) | type | ((DP >> 3) << 17) | ((kRows >> 4) << 24) | kIdescBMnMajor;
        const uint64_t k_desc = smem_desc_sw128(0), v_desc = smem_desc_mn_sw128(0, kTok * 128);
        const uint32_t k_lo = (uint32_t)k_desc, k_hi = (uint32_t)(k_desc >> 32);
        const uint32_t v_lo = (uint32_t)v_desc, v_hi = (uint32_t)(v_desc >> 32);
        const uint32_t ring_a = smem_u32(ring) >> 4, q_a = k_lo + ((smem_u32(q_s) + m * S::Q_TILE) >> 4);
        int q_uses = 0, slot = 0;
        uint32_t full_phase = 0;
        int64_t k_no = 0;              // tiles multiplied with P
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, p.wait_ns, abort_flag, p.status, kCodeTreeMma));
            if (ok) tc_fence_after();
            return ok;
        };
        auto next_slot = [&]() {
            if (++slot == NS) slot = 0, full_phase ^= 1;
        };
        // S of tile k into buffer k & 1, from the K in `slot`.  The buffer held the P of two tiles ago: that product was
        // issued before, and one thread's instructions run in order.
        bool live = true;              // there are rows among the 128; where not, the barriers alone are served
        auto scores = [&](int64_t k) {
            const uint32_t b = k_lo + ring_a + slot * (S::SLOT >> 4), d = tmem + (m * 2 + (int)(k & 1)) * kTok;
            if (elected()) {
                if (live)
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j) {
                        const uint32_t qj = ((j / 4) * kRows * 128 + (j % 4) * 32) >> 4;
                        const uint32_t kj = ((j / 4) * kTok * 128 + (j % 4) * 32) >> 4;
                        if (j == 0)
                            mma_ss<false>(d, q_a + qj, b + kj, k_hi, idesc_s);
                        else
                            mma_ss<true>(d, q_a + qj, b + kj, k_hi, idesc_s);
                    }
                tc_commit(s_full(m, (int)(k & 1)));
                tc_commit(empty(slot));
            }
            __syncwarp();
            next_slot();
        };
        for (Walk w = start; ok && w.u < w.end;) {
            const int32_t T = w.tiles();
            if (!wait(q_full(m), q_uses++ & 1)) break;
            live = MT == 1 || w.row.count > m * kRows;
            for (int i = 0; i < min(T, 2) && wait(full(slot), full_phase); ++i) scores(k_no + i);
            for (int32_t it = 0; ok && it < T; ++it, ++k_no) {
                const int buf = (int)(k_no & 1);
                // P, V and the K of two tiles on, which follows V in the ring, a lane each: one wait after another
                // would cost 200 cycles a piece
                const bool wrap = slot + 1 == NS;
                uint32_t bar = p_ready(m, buf), parity = (uint32_t)(k_no >> 1) & 1;
                if (lane == 1) bar = full(slot), parity = full_phase;
                if (lane == 2 && it + 2 < T) bar = full(wrap ? 0 : slot + 1), parity = wrap ? full_phase ^ 1 : full_phase;
                if (!wait(bar, parity)) break;
                const uint32_t a = tmem + (m * 2 + buf) * kTok, d = tmem + S::O_COL + m * DP;
                const uint32_t b = v_lo + ring_a + slot * (S::SLOT >> 4);
                if (elected()) {
                    if (live)
#pragma unroll
                        for (int j = 0; j < 2 * kTok / 16; ++j)  // the first numbers, then the second ones
                            mma_ts(d, a + j * 8, b + ((j % 4) * 2048 >> 4), v_hi, idesc_o, j > 0 ? 1u : it > 0);
                    tc_commit(pv_done(m, buf));
                    tc_commit(empty(slot));
                }
                __syncwarp();
                next_slot();
                if (it + 2 < T) scores(k_no + 2);
            }
            w.next(T);
        }
        // every instruction issued has completed once this wait is over
        if (elected()) tc_commit(all_done(m));
        __syncwarp();
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(all_done(m), 0)) {
            if (globaltimer() - t0 > p.wait_ns) break;
        }
        __syncwarp();
    } else if (warp < 4 * MT) {
        // ------------------------------------------------------------ softmax: a row per thread
        const int m = warp / 4, r = threadIdx.x;                 // row of the plane's tile
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t o_t = tmem + S::O_COL + m * DP + lanes;
        int64_t k_no = 0;
        bool first_seg = true, ok = true;
        int tile_no = 0, v_slot = 0;
        uint32_t v_phase = 0;
        for (Walk w = start; ok && w.u < w.end;) {
            const TreeRow row = w.row;
            const int32_t T = w.tiles(), new0 = row.len - row.n, h = w.h, t0 = w.t;
            const bool mine = r < row.count, some = (r & ~31) < row.count;
            const uint32_t rr = (uint32_t)((int64_t)row.plane * R + r);
            const int32_t i = mine ? (int32_t)sbt_div(p.group, rr) : 0, g = mine ? (int32_t)(rr - i * p.group.d) : 0;
            const int64_t q_row = row.q0 + i;
            float ref = -CUDART_INF_F, l = 0.f;
            // ---- this row's query (the last segment's is not read any more); zeros in rows that are not there
            {
                const char* const a = p.q + (q_row * p.ld_q + (int64_t)(h * (int32_t)p.group.d + g) * p.ld_qh) * 2;
                uint8_t* const to = q_s + m * S::Q_TILE + (r & 127) * 128;
                if (p.q_vec) {
                    constexpr int BATCH = DP / 8 % 16 == 0 ? 16 : 8;  // all loads of a row of 128 elements are on their way at once
#pragma unroll
                    for (int e0 = 0; e0 < DP / 8; e0 += BATCH) {
                        uint4 v[BATCH];
#pragma unroll
                        for (int e = 0; e < BATCH; ++e)
                            v[e] = mine && (e0 + e) * 8 < p.head_dim ? sbt_ld(reinterpret_cast<const uint4*>(a) + e0 + e)
                                                                     : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int e = 0; e < BATCH; ++e)
                            *reinterpret_cast<uint4*>(to + ((e0 + e) / 8) * kRows * 128 + (((e & 7) ^ (r & 7)) << 4)) = v[e];
                    }
                } else {
                    for (int d = 0; d < DP; ++d)
                        *reinterpret_cast<uint16_t*>(to + (d >> 6) * kRows * 128 + (((d >> 3 & 7) ^ (r & 7)) << 4) + (d & 7) * 2) =
                            mine && d < p.head_dim ? sbt_ld(reinterpret_cast<const uint16_t*>(a) + d) : (uint16_t)0;
                }
                fence_proxy_async_smem();
                mbar_arrive(q_full(m));
            }
            // bit j: this row sees position j of the tile (if it is on a page)
            auto sees = [&](int32_t pos0) -> uint64_t {
                const int64_t j0 = (int64_t)pos0 - new0;         // the new token at the tile's first position
                uint64_t bits = 0;
                if (p.mask) {
                    const uint32_t* const a = p.mask + q_row * p.ld_mask;
                    const int64_t w0 = j0 >> 5;
                    auto word = [&](int64_t x) -> uint64_t { return mine && x >= 0 && x < p.ld_mask ? sbt_ld(a + x) : 0u; };
                    const int sh = (int)(j0 & 31);
                    bits = (word(w0) | word(w0 + 1) << 32) >> sh;
                    if (sh) bits |= word(w0 + 2) << (64 - sh);
                } else if (i >= j0) {
                    bits = i - j0 >= 63 ? ~0ull : (2ull << (i - j0)) - 1;
                }
                if (j0 < 0) bits = j0 <= -64 ? ~0ull : bits | ((1ull << -j0) - 1);
                const int64_t left = row.n - j0;                 // positions up to the sequence's end
                if (left < 64) bits &= left <= 0 ? 0 : (1ull << left) - 1;
                return bits;
            };
            // the ring's slots go to K K V K V .. K V V
            v_slot += T > 1 ? 2 : 1;
            if (v_slot >= NS) v_slot -= NS, v_phase ^= 1;
            for (int32_t it = 0; it < T; ++it, ++k_no) {
                const int buf = (int)(k_no & 1);
                if (!mbar_wait_bounded(s_full(m, buf), (uint32_t)(k_no >> 1) & 1, p.wait_ns, abort_flag, p.status, kCodeTreeSoft))
                    ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t on_page = s_bits[tile_no++ & (kBits - 1)];
                if (some) {
                    const uint32_t s_t = tmem + (m * 2 + buf) * kTok + lanes;
                    uint32_t x[2][32];
                    tmem_ld_32x32b_x32(s_t, x[0]);
                    tmem_ld_32x32b_x32(s_t + 32, x[1]);
                    tmem_ld_wait();
                    const int32_t pos0 = (t0 + it) * kTok;
                    if (p.negate)
#pragma unroll
                        for (int j = 0; j < 64; ++j) x[j / 32][j % 32] ^= 0x80000000u;
                    if (on_page != ~0ull || pos0 + kTok > new0) {
                        const uint64_t vis = on_page & sees(pos0);
                        const uint32_t seen[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (!(seen[j / 32] >> j % 32 & 1)) x[j / 32][j % 32] = 0xff800000u;
                    }
                    float top[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int j = 0; j < 64; j += 2)
                        top[j / 2 & 3] = max3(top[j / 2 & 3], __uint_as_float(x[j / 32][j % 32]), __uint_as_float(x[j / 32][j % 32 + 1]));
                    float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    if (most != -CUDART_INF_F) most *= p.scale;
                    const bool take = most > ref + S::SLACK;     // ref = -inf: as soon as anything is seen
                    if (__any_sync(0xffffffffu, take)) {
                        const float f = take ? sbt_attn::exp2_fast(ref - most) : 1.f;
                        if (take) ref = most;
                        l *= f;
                        if (it > 0) {
                            if (!mbar_wait_bounded(pv_done(m, buf ^ 1), (uint32_t)((k_no - 1) >> 1) & 1, p.wait_ns, abort_flag,
                                                   p.status, kCodeTreeSoft))
                                ok = false;
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int d = 0; d < DP; d += 32) {
                                uint32_t o[32];
                                tmem_ld_32x32b_x32(o_t + d, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st_x32(o_t + d, o);
                            }
                        }
                    }
                    const float base = ref == -CUDART_INF_F ? 0.f : S::SHIFT - ref;
                    float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {  // 16 scores at a time: their registers are free for what comes after
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int k = c * 16 + 2 * j;
                            const float2 y = fma2(make_float2(__uint_as_float(x[k / 32][k % 32]), __uint_as_float(x[k / 32][k % 32 + 1])),
                                                  make_float2(p.scale, p.scale), make_float2(base, base));
                            const float2 e = make_float2(sbt_attn::exp2_fast(y.x), sbt_attn::exp2_fast(y.y));
                            sum[j & 1] = add2(sum[j & 1], e);
                            hi[j] = pack2<KIND>(e.x, e.y);
                            const float2 d = add2(e, unpack2<KIND>(hi[j] ^ 0x80008000u));
                            lo[j] = pack2<KIND>(d.x, d.y);
                        }
                        tmem_st_x8(s_t + c * 8, hi);
                        tmem_st_x8(s_t + 32 + c * 8, lo);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_st_wait();
                }
                if ((t0 + it + 1) * kTok > new0) {
                    // the tile holds new positions, or ends past the last: infinities and NaN of the former and all
                    // of what follows become zero in V
                    const int s = v_slot;
                    if (!mbar_wait_bounded(full(s), v_phase, p.wait_ns, abort_flag, p.status, kCodeTreeSoft)) ok = false;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int32_t pos = (t0 + it) * kTok + (r & 127) / 2;
                    if (pos >= new0) {
                        uint8_t* const x = ring + s * S::SLOT + (r & 127) / 2 * 128;
                        const uint32_t e = KIND == kBF16 ? 0x7F807F80u : 0x7C007C00u;
                        for (int c = (r & 1) * (DP / 16); c < ((r & 1) + 1) * (DP / 16); ++c) {
                            uint4* const at = reinterpret_cast<uint4*>(x + (c >> 3) * kTok * 128 + (((c & 7) ^ ((r & 127) / 2 & 7)) << 4));
                            uint4 v = *at;
                            uint32_t* const word = reinterpret_cast<uint32_t*>(&v);
                            bool found = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t keep = pos >= row.len ? 0u : __vcmpne2(word[k] & e, e);
                                found |= (word[k] & ~keep) != 0;
                                word[k] &= keep;
                            }
                            if (found) {
                                if (pos < row.len) *s_special = 1;
                                *at = v;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                v_slot += it + 2 < T ? 2 : 1;  // K of two tiles on follows in the ring
                if (v_slot >= NS) v_slot -= NS, v_phase ^= 1;
                tc_fence_before();
                mbar_arrive(p_ready(m, buf));
            }
            if (!ok) break;
            // ---- the segment's state, once the last product is done
            if (!mbar_wait_bounded(pv_done(m, (int)(k_no - 1) & 1), (uint32_t)((k_no - 1) >> 1) & 1, p.wait_ns, abort_flag,
                                   p.status, kCodeTreeSoft))
                ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const bool ends = t0 + T == row.tiles, cut = t0 != 0, whole = ends && !cut;
            const int32_t qh = h * (int32_t)p.group.d + g;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (first_seg ? 0 : 1);
            const float m_out = ref == -CUDART_INF_F ? ref : ref - S::SHIFT, inv = sbt_attn::inverse(l);
            if (some) {
                if (mine && whole && p.lse) p.lse[q_row * p.q_heads + qh] = sbt_attn::log_sum(m_out, l);
                if (mine && !whole) p.part_ml[slot * R + r] = make_float2(m_out, l);
                const bool poison = *s_special != 0;
#pragma unroll 1
                for (int d = 0; d < DP; d += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(o_t + d, o);
                    tmem_ld_wait();
                    if (!mine) continue;
                    if (whole)
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
                    if (poison) {
                        // what was taken out of the new positions' values goes to the rows that see it
                        for (int32_t pos = max(max(new0, 0), t0 * kTok); pos < min((t0 + T) * kTok, row.len); ++pos) {
                            if (!(sees(pos) & 1)) continue;
                            const uint32_t pg = sbt_div(p.page_size, (uint32_t)pos);
                            const int32_t page = sbt_ld(p.table + (int64_t)row.seq * p.ld_table + pg);
                            if (page < 0 || page >= p.n_pages) continue;
                            const uint16_t* const v = reinterpret_cast<const uint16_t*>(p.v) + page * p.ld_page +
                                (int64_t)(pos - (int32_t)(pg * p.page_size.d)) * p.ld_slot + h * p.ld_head;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (d + j < p.head_dim) {
                                    const uint16_t e = sbt_ld(v + d + j);
                                    if (special<KIND>(e)) o[j] = __float_as_uint(__uint_as_float(o[j]) + Num<KIND>::get(e));
                                }
                        }
                    }
                    if (!whole) {
                        float4* const to = p.part_o + (slot * (DP / 4) + d / 4) * R + r;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            to[j * R] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
                    } else {
                        uint16_t* const to = reinterpret_cast<uint16_t*>(p.out) + q_row * p.ld_out + qh * p.ld_oh + d;
                        if (p.out_vec) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (d + 8 * j < p.head_dim) {
                                    uint32_t y[4];
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        y[k] = pack2<KIND>(__uint_as_float(o[8 * j + 2 * k]), __uint_as_float(o[8 * j + 2 * k + 1]));
                                    reinterpret_cast<uint4*>(to)[j] = make_uint4(y[0], y[1], y[2], y[3]);
                                }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (d + j < p.head_dim) to[j] = Num<KIND>::put(__uint_as_float(o[j]));
                        }
                    }
                }
            }
            tc_fence_before();
            if (!cut && threadIdx.x == 0) {
                TreeDesc e = {};
                if (!whole) {
                    e.valid = 1, e.b = row.b, e.h = h, e.plane = row.plane, e.first = c, e.first_slot = first_seg ? 0 : 1;
                    e.last = line.warp_of(w.u - t0 + row.tiles - 1);
                }
                if (p.desc_by_line)
                    p.desc[((int64_t)row.b * p.kv_heads + h) * p.planes + row.plane] = e;
                else if (e.valid)
                    p.desc[blockIdx.x] = e;
            }
            first_seg = false;
            w.next(T);
        }
    }

    // ---- planes that hold no position they could see: zeros, and a log-sum-exp of minus infinity
    if (warp == 4 * MT)  // (the first warp of the copies is done before the others)
        for (int64_t b = c; b < p.batch; b += gridDim.x) {
            TreeRow row = row_of(p, (int32_t)b, R);
            for (int32_t i = 0; i < p.planes; ++i) {
                set_plane(p, row, i, R);
                if (row.tiles) continue;
                if (p.desc_by_line)
                    for (int32_t h = lane; h < p.kv_heads; h += 32) p.desc[((int64_t)b * p.kv_heads + h) * p.planes + i].valid = 0;
                else if (row.count == 0)
                    break;
                for (int64_t e = lane; e < (int64_t)row.count * p.kv_heads; e += 32) {
                    const int32_t h = (int32_t)(e / row.count);
                    const uint32_t rr = (uint32_t)((int64_t)i * R + e - (int64_t)h * row.count), tok = sbt_div(p.group, rr);
                    const int32_t qh = h * (int32_t)p.group.d + (int32_t)(rr - tok * p.group.d);
                    uint16_t* const to = reinterpret_cast<uint16_t*>(p.out) + (row.q0 + (int64_t)tok) * p.ld_out + qh * p.ld_oh;
                    for (int d = 0; d < p.head_dim; ++d) to[d] = 0;
                    if (p.lse) p.lse[(row.q0 + (int64_t)tok) * p.q_heads + qh] = -CUDART_INF_F;
                }
            }
        }
    tc_fence_before();
    __syncthreads();
    if (TMA && *abort_flag && warp == 4 * MT)  // copies in flight land before the block leaves
        for (int i = 0; i < NS; ++i) {
            const uint64_t t0 = globaltimer();
            while (s_uses[i] > 0 && !mbar_try_wait(full(i), (s_uses[i] - 1) & 1) && globaltimer() - t0 < p.wait_ns) {
            }
        }
    if (*abort_flag && p.desc_by_line && threadIdx.x == 0 && !idle)
        for (Walk w = start; w.u < w.end; w.next(w.tiles()))  // what was not finished is not joined
            if (w.t == 0) p.desc[((int64_t)w.row.b * p.kv_heads + w.h) * p.planes + w.row.plane].valid = 0;
    if (warp == WARPS - 1) {
        tc_fence_after();
        tmem_dealloc(tmem, S::COLS);
    }
}

// Adds the parts of cut lines in the order of the line.  A block takes 32 rows, a lane each, of one of them, and its
// eight warps 8 / groups vectors of four elements, whose parts `groups` warps share out and join in shared memory.
// Latency bounds it: a pass over the parts' maxima ahead of the parts themselves cost 2 us of the 41 of one tree's call.
template <int KIND, int DP, int MT>
__global__ void __launch_bounds__(kJoin) k_tree_join(const TreeAttnParams p, int32_t pieces, int32_t groups) {
    constexpr int R = MT * kRows;
    __shared__ float4 s_o[kJoin];
    __shared__ float s_l[kJoin], s_top[kJoin];
    griddep_wait();
    const TreeDesc e = p.desc[blockIdx.x / pieces];
    if (!e.valid) return;
    TreeRow row = row_of(p, e.b, R);
    set_plane(p, row, e.plane, R);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quads = kJoin / 32 / groups, rest = blockIdx.x % pieces;
    const int r0 = rest / (DP / 4 / quads) * 32, quad = rest % (DP / 4 / quads) * quads + warp / groups, group = warp % groups;
    if (r0 >= row.count) return;
    const int r = min(r0 + lane, row.count - 1);
    auto slot = [&](int32_t i) -> int64_t { return 2ll * (e.first + i) + (i == 0 ? e.first_slot : 0); };
    const int32_t n = e.last - e.first + 1;
    float top = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int BATCH = 8;  // parts on their way at once
    for (int32_t first = group; first < n; first += BATCH * groups) {
        float2 ml[BATCH];
        float4 x[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int32_t i = first + j * groups;
            ml[j] = make_float2(-CUDART_INF_F, 0.f), x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i >= n) continue;
            ml[j] = sbt_ld(p.part_ml + slot(i) * R + r);
            x[j] = sbt_ld(p.part_o + (slot(i) * (DP / 4) + quad) * R + r);
        }
        const float was = top;
#pragma unroll
        for (int j = 0; j < BATCH; ++j) top = fmaxf(top, ml[j].x);
        const float ts = top == -CUDART_INF_F ? 0.f : top, f = sbt_attn::exp2_fast(was - ts);
        l *= f, o[0] *= f, o[1] *= f, o[2] *= f, o[3] *= f;
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const float a = sbt_attn::exp2_fast(ml[j].x - ts);
            l += ml[j].y * a;
            o[0] += x[j].x * a, o[1] += x[j].y * a, o[2] += x[j].z * a, o[3] += x[j].w * a;
        }
    }
    s_o[threadIdx.x] = make_float4(o[0], o[1], o[2], o[3]);
    s_l[threadIdx.x] = l;
    s_top[threadIdx.x] = top;
    __syncthreads();
    // neighbouring threads write neighbouring vectors of a row
    const int mine = threadIdx.x / quads, q = threadIdx.x % quads;
    if (threadIdx.x >= 32 * quads || r0 + mine >= row.count) return;
    l = 0.f, o[0] = o[1] = o[2] = o[3] = 0.f, top = -CUDART_INF_F;
    for (int i = 0; i < groups; ++i) top = fmaxf(top, s_top[(q * groups + i) * 32 + mine]);
    const float ts = top == -CUDART_INF_F ? 0.f : top;
    for (int i = 0; i < groups; ++i) {
        const int from = (q * groups + i) * 32 + mine;
        const float4 x = s_o[from];
        const float a = sbt_attn::exp2_fast(s_top[from] - ts);
        l += s_l[from] * a;
        o[0] += x.x * a, o[1] += x.y * a, o[2] += x.z * a, o[3] += x.w * a;
    }
    const uint32_t rr = (uint32_t)((int64_t)e.plane * R + r0 + mine), i = sbt_div(p.group, rr);
    const int32_t qh = e.h * (int32_t)p.group.d + (int32_t)(rr - i * p.group.d), d = (quad - warp / groups + q) * 4;
    const int64_t q_row = row.q0 + (int64_t)i;
    const float inv = sbt_attn::inverse(l);
    uint16_t* const to = reinterpret_cast<uint16_t*>(p.out) + q_row * p.ld_out + qh * p.ld_oh + d;
    if (p.out_vec && d + 4 <= p.head_dim) {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack2<KIND>(o[0] * inv, o[1] * inv), pack2<KIND>(o[2] * inv, o[3] * inv));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (d + j < p.head_dim) to[j] = Num<KIND>::put(o[j] * inv);
    }
    if (d == 0 && p.lse) p.lse[q_row * p.q_heads + qh] = sbt_attn::log_sum(top, l);
}

template <int KIND, int DP, int MT, bool TMA>
sbt_status enqueue(sbt_context* ctx, TreeAttnParams& p, const TreeMaps& maps, void* workspace, cudaStream_t stream) {
    typedef TreeShape<KIND, DP, MT, TMA> S;
    // (the runtime's count of resident blocks is one for any kernel that allocates TMEM)
    sbt_resident_blocks<k_tree_attention<KIND, DP, MT, TMA>>(ctx, S::THREADS, S::SMEM);
    const int resident = ctx->sm_count * S::BLOCKS;
    p.planes = (int32_t)sbt_cdiv((int64_t)p.max_new * p.group.d, S::R);
    const int64_t blocks = resident, lines = (int64_t)p.batch * p.kv_heads * p.planes;
    p.desc_by_line = lines <= blocks;
    p.desc = (TreeDesc*)workspace;
    p.part_ml = (float2*)((char*)workspace + sbt_cdiv(blocks * sizeof(TreeDesc), 256) * 256);
    p.part_o = (float4*)(p.part_ml + 2 * blocks * S::R);
    sbt_status st = sbt_cuda_check(sbt_launch_dependent(k_tree_attention<KIND, DP, MT, TMA>, dim3((unsigned)blocks),
                                                        dim3(S::THREADS), S::SMEM, stream, p, maps.k, maps.v),
                                   "paged_tree_attention launch");
    if (st || (st = sbt_after_launch(ctx, "paged_tree_attention"))) return st;
    const int64_t n_desc = p.desc_by_line ? lines : blocks;
    // Few lines are cut into many parts: four warps share a vector's; many lines into two or three.
    const int64_t row_groups = sbt_cdiv(std::min<int64_t>(S::R, (int64_t)p.max_new * p.group.d), 32);
    const int32_t groups = n_desc * row_groups * (DP / 32) < 4 * ctx->sm_count ? 4 : 1;
    const int32_t pieces = (int32_t)(row_groups * (DP / 4) / (kJoin / 32 / groups));
    st = sbt_cuda_check(sbt_launch_dependent(k_tree_join<KIND, DP, MT>, dim3((unsigned)(n_desc * pieces)), dim3(kJoin), 0,
                                             stream, p, pieces, groups),
                        "paged_tree_attention join launch");
    if (st) return st;
    return sbt_after_launch(ctx, "paged_tree_attention join");
}

template <int KIND, int DP, int MT>
sbt_status enqueue(sbt_context* ctx, TreeAttnParams& p, const TreeMaps& maps, void* workspace, cudaStream_t stream) {
    return maps.use ? enqueue<KIND, DP, MT, true>(ctx, p, maps, workspace, stream)
                    : enqueue<KIND, DP, MT, false>(ctx, p, maps, workspace, stream);
}

// One translation unit each: the head sizes to 128 and those past it.
template <int KIND> sbt_status narrow(sbt_context*, TreeAttnParams&, const TreeMaps&, bool two, void* workspace, cudaStream_t);
template <int KIND> sbt_status wide(sbt_context*, TreeAttnParams&, const TreeMaps&, void* workspace, cudaStream_t);

}  // namespace sbt_tree
