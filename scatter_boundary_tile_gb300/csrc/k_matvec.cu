// A few rows times a matrix of 4-bit weights with group scales:
//   y[t][n] = alpha sum_k x[t][k] w[k][n] s[k / group][n],
// w in E2M1, two columns a byte, s in E8M0 or E4M3.
//
// The weights are read once and bound the call: 0.5 byte each, so at the copy
// rate an SM has to turn ~47 of them a clock into numbers and multiply them for
// up to 16 rows.  The products run on mma.sync m16n8k16 (fp16 in, fp32 sums):
// 16 columns of w by 8 rows of x, 16 k.  E2M1 is exact in fp16 and has a
// conversion of two codes at once; a tcgen05 tile in fp16 would want the weights
// in shared memory, written there by the same instructions and read again.  (One of
// E2M1 codes with block scales and x as a sum of E4M3 codes has not been tried.)
//
// A column's neighbour lies in the same byte, but the conversion and the matrix
// instruction want pairs along k: two bytes of rows k and k + 1 trade nibbles
// (4 operations for 16 weights), the even column's pair to row g of the tile
// and the odd column's to row g + 8.  The k of a step are numbered so that a
// lane's four are neighbours, for the weights and for x alike.
//
// Groups.  The products of U k (32, or 16) are summed by the matrix unit and
// added to the running sums times the group's scale.  A stage holds 64 k where
// they are whole groups or part of one, so that waits, copies and addresses are
// paid once for them.
//
// x.  fp16 enters as it is.  bf16 and fp32 are scaled by a power of two to
// below 2^15, per row and for the k seen so far (as the running maximum of a
// softmax: when it grows, the sums are scaled), and enter as one and two fp16
// numbers; bf16's 8 bits fit in fp16's 11 unless they are below its last step,
// 2^-39 of the largest.
//
// Split.  A block has 256 columns and a share of k; its warps take 128 columns and
// a share of that k (with 256 columns the sums leave no registers for what is on
// its way).  Every warp has a private ring of stages filled by cp.async and waits
// for no other until the end.  A cluster of up to eight blocks shares the k of one
// tile; warps, then blocks, join in a fixed order through shared memory.
//
// LINE.  For 9 to 16 tokens the sums take 64 registers a lane, and twelve warps an
// SM have none left for stages of 64 k.  Eight warps do, and where there are many
// columns they go from tile to tile of 128: the copies of the next tile are on
// their way while a tile's sums pass from warp to warp through one buffer, so that
// no block starts and ends without work.  (16 tokens bf16, 131072 x 4096: 151 us by
// blocks of twelve warps, 118 so; blocks of eight warps 155.  Up to 8 tokens the
// two are equal, and there is only the first.)
//
// Measured (GB300), weights at copy rate in brackets: 1 token bf16, 4096 x 4096
// 8.3 us (1.3: launch, first copies and two joins are its time), 5 tokens fp16,
// 28672 x 8192 with E4M3 scales per 16 41 us (19.5), 8 tokens fp16, 131072 x 4096
// 71 us (43), 16 tokens fp16 99, bf16 118, with unaligned scales 123; fp32 x, 65536 x
// 4096, 1 and 8 tokens 58 us (21; bf16 42), 16 tokens 105 (bf16 70).  The ALU pipe
// (50 to 60 % busy) and dependent instructions bound the large ones: 21
// instructions for 256 weights with 8 tokens, 32 with 16 of bf16.
#include <algorithm>

#include "matvec_copies.h"
#include "sbt_internal.cuh"
#include "sbt_num.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace sbt_num;
using sbt_ptx::griddep_wait;

constexpr int kCols = 256, kClusterMost = 8;
constexpr int kPitch = kCols + 20;  // floats between rows of partial sums: lanes of a half warp meet no bank twice
constexpr int kFixedRows = 128;     // what a block costs besides its k, in k of a warp
constexpr int kLineRows = 144;      // the same of a tile, and of a call, where blocks go from tile to tile

struct MatvecParams {
    const char* x;
    const uint8_t *w, *s;
    char* y;
    int64_t ld_x, ld_w, ld_s, ld_y;  // bytes
    int64_t tokens, N, K, group;
    float alpha;
    int32_t y_kind, ranks, x_vec;
    int64_t items;               // LINE: tiles times eights (or sixteens) of tokens
    int32_t chunks;
};

// U: k whose products are summed before they are scaled; SU: such units of a stage.
template <int U, int SU, int MT, bool ALIGNED, bool LINE>
struct Shape {
    static constexpr int ROWS = U * SU;
    // 16 rows of x: the sums fill twice the registers, and twelve (LINE: eight) warps an SM take the place of sixteen
    static constexpr int BLOCKS = MT == 1 ? 2 : 1, WARPS = MT == 1 || LINE ? 8 : 12;
    static constexpr int CW = 128, COLS = LINE ? CW : kCols, KW = WARPS * CW / COLS;  // columns of a warp and a block, warps along k
    static constexpr int LANE = CW / 16;                   // bytes of a row that a lane takes
    static constexpr int PITCH = ALIGNED ? CW / 2 : CW / 2 + 16;  // bytes of a row of weights in a stage
    static constexpr int SCALES = CW + 32;                 // a row of scales, from the 16-byte boundary before it
    static constexpr int STAGE = ROWS * PITCH + SU * SCALES;
    static constexpr int CHAIN = LINE ? MT * 8 * 33 * 16 : 0;  // the running sums of a tile, 16 bytes of a lane beside another's
    static constexpr int MOST = ((220 << 10) - CHAIN) / (BLOCKS * WARPS * STAGE), STAGES = MOST < 8 ? MOST : 8;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int PART = 8 * kPitch * 4;            // sums of 256 columns
    static constexpr size_t SMEM = LINE ? (size_t)WARPS * RING + CHAIN
                                        : (size_t)WARPS * RING > (size_t)KW * PART ? (size_t)WARPS * RING : (size_t)KW * PART;
    // Place of byte `c` of row r (aligned rows): lanes that read together, their rows U / 4 apart, meet no bank twice.
    static __device__ __forceinline__ int place(int r, int c) {
        const int key = r / (U / 4) & 3;
        return (r ^ (key & 1)) * 64 + (c ^ (key << 4));
    }
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

// c = a b (+ c).
template <bool ADD>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (ADD)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A warp waits for the one before it, and lets the one after it go on (barriers of two warps).
__device__ __forceinline__ void chain_wait(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void chain_pass(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); }

// KIND: of x.  MT: 8 rows of x each.  LINE: a block goes from tile to tile.
template <int KIND, int U, int SU, bool E4M3, int MT, bool ALIGNED, bool LINE>
__global__ void __launch_bounds__(32 * Shape<U, SU, MT, ALIGNED, LINE>::WARPS, Shape<U, SU, MT, ALIGNED, LINE>::BLOCKS)
    k_matvec(const MatvecParams p) {
    typedef Shape<U, SU, MT, ALIGNED, LINE> S;
    typedef typename Num<KIND>::T T;
    constexpr int WORDS = S::LANE / 4, TILES = 4 * WORDS;  // of a lane's piece of a row; matrix tiles of a warp
    constexpr int STEPS = U / 16, ROWS = S::ROWS, TERMS = KIND == kF32 ? 2 : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int rank = LINE ? 0 : blockIdx.x % p.ranks;
    const int64_t stages = p.K / ROWS, items = LINE ? p.items : 1;
    // This warp's stages, of every tile; and a tile's columns and tokens.
    const int64_t workers = LINE ? S::KW : (int64_t)S::KW * p.ranks, me = (int64_t)rank * S::KW + warp % S::KW;
    const int64_t u0 = stages * me / workers, u1 = stages * (me + 1) / workers;
    const int todo = (int)(u1 - u0);
    const int64_t first_item = LINE ? blockIdx.x : 0, step_item = LINE ? gridDim.x : 1;
    auto columns = [&](int64_t item) {
        return LINE ? item / p.chunks * S::COLS : (int64_t)(blockIdx.x / p.ranks) * S::COLS + warp / S::KW * S::CW;
    };
    auto tokens = [&](int64_t item) { return (LINE ? item % p.chunks : (int64_t)blockIdx.y) * 8 * MT; };
    uint8_t* const ring = smem + warp * S::RING;
    const uint32_t ring_u32 = sbt_ptx::smem_u32(ring);
    griddep_wait();

    // ---- copies: the warp's columns of a stage's rows and its group's scales, nothing past their ends
    constexpr int LPR = S::CW / 32;                       // lanes of a row, 16 bytes each
    const int copy_c = ALIGNED ? lane % LPR * 16 : lane % (2 * LPR) * 16, copy_r = lane / (ALIGNED ? LPR : 2 * LPR);
    // Rows of scales: one for `per` stages (of which `left` are still to come for the copies and for the sums), or
    // one for every unit of a stage.
    const bool each = p.group < ROWS;
    const int per = each ? 1 : (int)(p.group / ROWS), s_rows = each ? SU : 1;
    const bool s_aligned = (((uintptr_t)p.s | (uintptr_t)p.ld_s) & 15) == 0;
    int w_bytes, s_bytes, copy_bytes, copy_left, copy_todo;
    int64_t copy_item = first_item;
    const uint8_t *copy_w, *copy_s;
    const int64_t s_row = each ? u0 * SU : u0 / per;
    const int s_left = per - (int)(u0 - s_row * per);       // (not for `each`, whose `per` is one)
    auto copy_start = [&] {
        const int64_t n0 = columns(copy_item);
        w_bytes = sbt_matvec::bytes_of((p.N + 1) / 2, n0 / 2, S::CW / 2);
        s_bytes = sbt_matvec::bytes_of(p.N, n0, S::CW);
        copy_bytes = sbt_matvec::piece_of(w_bytes, 0, copy_c);
        copy_w = p.w + n0 / 2 + (u0 * ROWS + copy_r) * p.ld_w;
        copy_s = p.s + s_row * p.ld_s + n0;
        copy_left = each ? 1 : s_left, copy_todo = todo;
    };
    copy_start();
    // places of this lane's rows of a stage, less what rows STEP apart are apart: they repeat after four
    constexpr int STEP = 32 / LPR;
    uint32_t at_place[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at_place[i] = S::place(i * STEP + copy_r, copy_c) - i * STEP * 64;
    const int64_t w_step = STEP * p.ld_w;
    auto copy = [&](int stage) {  // the next stage's
        if (copy_todo == 0) {
            if (!LINE || todo == 0 || copy_item + step_item >= items) return;
            copy_item += step_item;
            copy_start();
        }
        --copy_todo;
        const uint32_t dst = ring_u32 + stage * S::STAGE;
        const uint8_t* src = copy_w;
        copy_w += ROWS * p.ld_w;
        if (ALIGNED) {
            if (copy_bytes) {
                src += copy_c;
#pragma unroll
                for (int i = 0; i < ROWS / STEP; ++i) {
                    copy16(dst + at_place[i % 4] + i * STEP * 64, src, copy_bytes);
                    src += w_step;
                }
            }
        } else {
            // one piece more than a row has covers it from the 16-byte boundary before it
#pragma unroll 4
            for (int i = 0; i < ROWS / (16 / LPR); ++i) {
                const int shift = (int)((uintptr_t)src & 15), bytes = sbt_matvec::piece_of(w_bytes, shift, copy_c);
                if (bytes) copy16(dst + (i * (16 / LPR) + copy_r) * S::PITCH + copy_c, src - shift + copy_c, bytes);
                src += (16 / LPR) * p.ld_w;
            }
        }
        if (s_aligned) {
            const int row = lane / 8, at = lane % 8 * 16, bytes = sbt_matvec::piece_of(s_bytes, 0, at);
            if (row < s_rows && bytes)
                copy16(dst + ROWS * S::PITCH + row * S::SCALES + at, copy_s + row * p.ld_s + at, bytes);
        } else {
            for (int row = 0; row < s_rows; ++row) {
                const uint8_t* const a = copy_s + row * p.ld_s;
                const int shift = (int)((uintptr_t)a & 15), bytes = sbt_matvec::piece_of(s_bytes, shift, lane * 16);
                if (bytes) copy16(dst + ROWS * S::PITCH + row * S::SCALES + lane * 16, a - shift + lane * 16, bytes);
            }
        }
        if (--copy_left == 0) copy_left = per, copy_s += s_rows * p.ld_s;
    };

    // ---- x: this lane's U / 4 neighbouring k of each unit, of rows tok0 + 8 m + g; the next stage's while this one is used
    constexpr int XK = U / 4;
    struct alignas(16) Raw {
        T v[XK];
    };
    const T* x_at[MT];
    int x_todo;
    int64_t x_item = first_item;
    auto x_start = [&] {
        const int64_t tok = tokens(x_item) + g;
        x_todo = todo;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            x_at[m] = tok + m * 8 < p.tokens
                          ? reinterpret_cast<const T*>(p.x + (tok + m * 8) * p.ld_x) + u0 * ROWS + t * XK : nullptr;
    };
    x_start();
    auto load_x = [&](Raw (&r)[SU][MT]) {
        if (x_todo == 0) {
            if (!LINE || todo == 0 || x_item + step_item >= items) return;
            x_item += step_item;
            x_start();
        }
        --x_todo;
#pragma unroll
        for (int q = 0; q < SU; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const T* const a = x_at[m] + q * U;
                if (!x_at[m]) {
                    r[q][m] = Raw{};
                } else if (p.x_vec) {
                    if constexpr (sizeof(T) * XK >= 16) {
#pragma unroll
                        for (int i = 0; i < (int)sizeof(T) * XK / 16; ++i)
                            reinterpret_cast<uint4*>(&r[q][m])[i] = sbt_ld(reinterpret_cast<const uint4*>(a) + i);
                    } else {
                        *reinterpret_cast<uint2*>(&r[q][m]) = sbt_ld(reinterpret_cast<const uint2*>(a));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < XK; ++i) r[q][m].v[i] = sbt_ld(a + i);
                }
            }
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (x_at[m]) x_at[m] += ROWS;
    };

    Raw raw[SU][MT];
    load_x(raw);
#pragma unroll 1
    for (int i = 0; i < S::STAGES - 1; ++i) {
        copy(i);
        copy_commit();
    }
    int stage = 0;
#pragma unroll 1
    for (int64_t item = first_item; item < items; item += step_item) {
        const int64_t n0 = columns(item), tok0 = tokens(item);
        const uint8_t* sum_s = p.s + s_row * p.ld_s + n0;
        int sum_left = each ? 1 : s_left;
        float sum[MT][TILES][4];  // columns g * 2 * TILES + 2 i, + 1; rows 2 t, + 1 of x
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[m][i][k] = 0.f;
        int exponent[MT];  // x of row g enters as x 2^-exponent
#pragma unroll
        for (int m = 0; m < MT; ++m) exponent[m] = -126;

#pragma unroll 1
        for (int n = todo; n > 0; --n) {
            copy_wait<S::STAGES - 2>();
            __syncwarp();
            copy(stage == 0 ? S::STAGES - 1 : stage - 1);
            copy_commit();

            // x as fp16 pairs along k
            uint32_t b[SU][STEPS][MT][TERMS][2];
            if constexpr (KIND == kF16) {
#pragma unroll
                for (int q = 0; q < SU; ++q)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int s = 0; s < STEPS; ++s) {
                            const uint2 v = reinterpret_cast<const uint2*>(&raw[q][m])[s];
                            b[q][s][m][0][0] = v.x, b[q][s][m][0][1] = v.y;
                        }
            } else {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    // exponent of the largest finite |x| of the row in this stage; magnitudes order as their bits do
                    uint32_t most = 0;
                    if constexpr (KIND == kBF16) {
#pragma unroll
                        for (int q = 0; q < SU; ++q)
#pragma unroll
                            for (int i = 0; i < XK / 2; ++i)
                                most = __vmaxu2(most, reinterpret_cast<const uint32_t*>(&raw[q][m])[i] & 0x7FFF7FFFu);
                        most = max(most & 0xFFFF0000u, most << 16);
                    } else {
#pragma unroll
                        for (int q = 0; q < SU; ++q)
#pragma unroll
                            for (int i = 0; i < XK; ++i) most = max(most, __float_as_uint(Num<KIND>::get(raw[q][m].v[i])) & 0x7fffffffu);
                    }
                    int top = (int)(most >> 23);
                    if (top == 255) {   // an infinity or NaN: the largest of the others
                        top = 0;
#pragma unroll 1
                        for (int q = 0; q < SU * XK; ++q) {
                            T one = 0;
#pragma unroll
                            for (int i = 0; i < SU * XK; ++i)
                                if (i == q) one = raw[i / XK][m].v[i % XK];
                            const int e = (int)(__float_as_uint(Num<KIND>::get(one)) >> 23) & 255;
                            top = max(top, e == 255 ? 0 : e);
                        }
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int want = max(top - 127 - 14, -126);
                    if (__any_sync(0xffffffffu, want > exponent[m])) {
                        // (2^-126 at least, for more: finite sums count for nothing then, and infinities stay what they are)
                        const int top_e = max(want, exponent[m]), gap = min(top_e - exponent[m], 126);
                        exponent[m] = top_e;
                        // the rows of the sums are 2 t and 2 t + 1, held by lanes 8 t and 8 t + 4
                        const float f0 = power(-__shfl_sync(0xffffffffu, gap, 8 * t));
                        const float f1 = power(-__shfl_sync(0xffffffffu, gap, 8 * t + 4));
#pragma unroll
                        for (int i = 0; i < TILES; ++i) {
                            sum[m][i][0] *= f0, sum[m][i][1] *= f1;
                            sum[m][i][2] *= f0, sum[m][i][3] *= f1;
                        }
                    }
                    const float f = power(-exponent[m]);
#pragma unroll
                    for (int q = 0; q < SU; ++q)
#pragma unroll
                        for (int i = 0; i < XK / 2; ++i) {
                            const float lo = Num<KIND>::get(raw[q][m].v[2 * i]) * f, hi = Num<KIND>::get(raw[q][m].v[2 * i + 1]) * f;
                            const __half2 h = __floats2half2_rn(lo, hi);
                            b[q][i / 2][m][0][i % 2] = *reinterpret_cast<const uint32_t*>(&h);
                            if constexpr (TERMS == 2) {
                                const float2 v = __half22float2(h);
                                // what the first number leaves; nothing of an infinity
                                const __half2 r = __floats2half2_rn(isinf(lo) ? 0.f : lo - v.x, isinf(hi) ? 0.f : hi - v.y);
                                b[q][i / 2][m][TERMS - 1][i % 2] = *reinterpret_cast<const uint32_t*>(&r);
                            }
                        }
                }
            }
            load_x(raw);

            const uint8_t* const st = ring + stage * S::STAGE;
#pragma unroll
            for (int q = 0; q < SU; ++q) {
                // weights: rows q U + t U / 4 + 4 s + r, a lane's WORDS words of each
                uint32_t w[STEPS][4][WORDS];
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = q * U + t * XK + 4 * s + r;
                        if (ALIGNED) {
                            const uint2 v = *reinterpret_cast<const uint2*>(st + S::place(row, g * S::LANE));
                            w[s][r][0] = v.x, w[s][r][1] = v.y;
                        } else {
                            const int shift = (int)((uintptr_t)(p.w + ((u1 - n) * ROWS + row) * p.ld_w + n0 / 2) & 15);
                            const uint32_t* const a =
                                reinterpret_cast<const uint32_t*>(st + row * S::PITCH + g * S::LANE + (shift & ~3));
                            uint32_t c = a[0];
#pragma unroll
                            for (int j = 0; j < WORDS; ++j) {
                                const uint32_t d = a[j + 1];
                                w[s][r][j] = __funnelshift_r(c, d, (shift & 3) * 8);
                                c = d;
                            }
                        }
                    }
                uint32_t sc[2 * WORDS];  // scales of its 8 WORDS columns
                {
                    const int row = each ? q : 0, shift = (int)((uintptr_t)(sum_s + row * p.ld_s) & 15);
                    const uint8_t* const a = st + ROWS * S::PITCH + row * S::SCALES + g * 2 * S::LANE;
                    if (shift == 0) {
                        const uint4 v = *reinterpret_cast<const uint4*>(a);
                        sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
                    } else {
                        const uint32_t* const at = reinterpret_cast<const uint32_t*>(a + (shift & ~3));
                        uint32_t c = at[0];
#pragma unroll
                        for (int j = 0; j < 2 * WORDS; ++j) {
                            const uint32_t d = at[j + 1];
                            sc[j] = __funnelshift_r(c, d, (shift & 3) * 8);
                            c = d;
                        }
                    }
                }
                // a byte of the last words may be past the scales and the weights: columns past N, which nobody reads
#pragma unroll
                for (int j = 0; j < WORDS; ++j) {
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
                            float c[4];
#pragma unroll
                            for (int s = 0; s < STEPS; ++s) {
                                const uint32_t frag[4] = {a[s][0][i], a[s][1][i], a[s][2][i], a[s][3][i]};
#pragma unroll
                                for (int v = 0; v < TERMS; ++v)
                                    if (s == 0 && v == 0)
                                        mma<false>(c, frag, b[q][s][m][v][0], b[q][s][m][v][1]);
                                    else
                                        mma<true>(c, frag, b[q][s][m][v][0], b[q][s][m][v][1]);
                            }
                            float(&d)[4] = sum[m][4 * j + i];
                            d[0] = fmaf(c[0], f.x, d[0]), d[1] = fmaf(c[1], f.x, d[1]);
                            d[2] = fmaf(c[2], f.y, d[2]), d[3] = fmaf(c[3], f.y, d[3]);
                        }
                    }
                }
            }
            if (--sum_left == 0) sum_left = per, sum_s += s_rows * p.ld_s;
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
        }
        // ---- from tile to tile: the warps add their sums to one buffer in their order, each when the one before it has; the
        // last writes y and lets the first go on.  (A warp passes again only after the next one has waited: all of them
        // have then added, and the last has let the first go on.)
        if constexpr (LINE) {
            float* const buf = reinterpret_cast<float*>(smem + S::WARPS * S::RING);
            if (warp > 0 || item != first_item) chain_wait(warp > 0 ? warp - 1 : S::KW - 1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float f0 = 1.f, f1 = 1.f;
                if (KIND != kF16) {
                    f0 = power(__shfl_sync(0xffffffffu, exponent[m], 8 * t));
                    f1 = power(__shfl_sync(0xffffffffu, exponent[m], 8 * t + 4));
                }
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    const float(&d)[4] = sum[m][i];
                    float4* const at = reinterpret_cast<float4*>(buf) + (m * 8 + i) * 33 + lane;
                    float4 v = make_float4(d[0] * f0, d[1] * f1, d[2] * f0, d[3] * f1);
                    if (warp > 0) {
                        const float4 w = *at;
                        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                    }
                    *at = v;
                }
            }
            __syncwarp();
            if (warp < S::KW - 1) {
                chain_pass(warp);
            } else {
#pragma unroll 1
                for (int r = 0; r < 8 * MT && tok0 + r < p.tokens; ++r) {
                    char* const y = p.y + (tok0 + r) * p.ld_y;
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = 32 * j + lane;
                        v[j] = p.alpha * buf[((r / 8 * 8 + c % 16 / 2) * 33 + c / 16 * 4 + r % 8 / 2) * 4 + c % 2 * 2 + r % 2];
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t n = n0 + 32 * j + lane;
                        if (n >= p.N) break;
                        if (p.y_kind == kF32)
                            reinterpret_cast<float*>(y)[n] = v[j];
                        else
                            reinterpret_cast<uint16_t*>(y)[n] = p.y_kind == kBF16 ? Num<kBF16>::put(v[j]) : Num<kF16>::put(v[j]);
                    }
                }
                __syncwarp();
                if (item + step_item < items) chain_pass(S::KW - 1);
            }
            continue;
        }
        copy_wait<0>();

        // ---- the warps' sums, then the blocks': a block finishes every p.ranks-th row
        const int64_t tile = blockIdx.x / p.ranks;
        float* const part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float f0 = 1.f, f1 = 1.f;
            if (KIND != kF16) {
                f0 = power(__shfl_sync(0xffffffffu, exponent[m], 8 * t));
                f1 = power(__shfl_sync(0xffffffffu, exponent[m], 8 * t + 4));
            }
            __syncthreads();
            // columns lie 34 floats apart for every 32 of the tile
            float* const mine = part + warp % S::KW * 8 * kPitch;
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                const int col = warp / S::KW * S::CW + g * 2 * TILES + 2 * i, n = (col >> 5) * 34 + (col & 31);
                const float(&d)[4] = sum[m][i];
                *reinterpret_cast<float2*>(mine + (2 * t) * kPitch + n) = make_float2(d[0] * f0, d[2] * f0);
                *reinterpret_cast<float2*>(mine + (2 * t + 1) * kPitch + n) = make_float2(d[1] * f1, d[3] * f1);
            }
            __syncthreads();
            const int n = threadIdx.x, at = (n >> 5) * 34 + (n & 31);  // the first 256 threads take a column each
            const bool adds = n < kCols;
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                v[r] = 0.f;
#pragma unroll
                for (int w = 0; w < S::KW && adds; ++w) v[r] += part[(w * 8 + r) * kPitch + at];
            }
            if (p.ranks > 1) {
                __syncthreads();
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (adds) part[r * kPitch + at] = v[r];
                sbt_ptx::cluster_sync();
            }
            auto put = [&](int r, float x) {
                const int64_t tok = tok0 + m * 8 + r;
                if (tok >= p.tokens || !adds || tile * kCols + n >= p.N) return;
                char* const y = p.y + tok * p.ld_y;
                x *= p.alpha;
                if (p.y_kind == kF32)
                    reinterpret_cast<float*>(y)[tile * kCols + n] = x;
                else
                    reinterpret_cast<uint16_t*>(y)[tile * kCols + n] = p.y_kind == kBF16 ? Num<kBF16>::put(x) : Num<kF16>::put(x);
            };
            if (p.ranks == 1) {
#pragma unroll
                for (int r = 0; r < 8; ++r) put(r, v[r]);
            } else {
                const uint32_t from = sbt_ptx::smem_u32(part + at);
                for (int r = rank; adds && r < 8 && tok0 + m * 8 + r < p.tokens; r += p.ranks) {
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
}

template <int KIND, int U, int SU, int SL, bool E4M3, int MT, bool ALIGNED>
sbt_status launch(sbt_context* ctx, MatvecParams& p, cudaStream_t stream) {
    constexpr auto kern = k_matvec<KIND, U, SU, E4M3, MT, ALIGNED, false>;
    typedef Shape<U, SU, MT, ALIGNED, false> S;
    const int64_t tiles = sbt_cdiv(p.N, kCols), chunks = sbt_cdiv(p.tokens, 8 * MT), stages = p.K / S::ROWS;
    // Blocks per tile: the number with which the last wave's end comes first.  (Clusters are counted as they fit groups of
    // SMs: by blocks alone 16 tiles of 16 tokens took eight each, 22 us instead of 15.)
    int64_t best = INT64_MAX;
    for (int c = 1; c <= kClusterMost && (c == 1 || c * S::KW <= stages); ++c) {
        const int64_t waves = sbt_cdiv(tiles * chunks, sbt_resident_clusters<kern>(ctx, 32 * S::WARPS, S::SMEM, c));
        const int64_t cost = waves * (sbt_cdiv(stages, (int64_t)c * S::KW) * S::ROWS + kFixedRows);
        if (cost < best) best = cost, p.ranks = c;
    }
    if constexpr (ALIGNED && MT == 2) {
        // A row of k of 128 columns costs a warp 1.8 times as long among twelve as among eight with two units a stage, and
        // 1.4 times as long with one.  16 tokens bf16, K 4096, by blocks and from tile to tile: N 8192 16 and 21 us, 16384
        // 24 and 21, 28672 36 and 37, 40960 70 and 52, 100000 112 and 103; K 2048, N 20000 22 and 25.
        constexpr auto line = k_matvec<KIND, U, SL, E4M3, MT, true, true>;
        typedef Shape<U, SL, MT, true, true> L;
        p.items = sbt_cdiv(p.N, L::COLS) * chunks, p.chunks = (int32_t)chunks;
        const int blocks = sbt_resident_blocks<line>(ctx, 32 * L::WARPS, L::SMEM);
        const int64_t waves = sbt_cdiv(p.items, blocks);
        const int64_t cost = waves * (sbt_cdiv(p.K / L::ROWS, L::KW) * L::ROWS + kLineRows) + kLineRows;
        if (cost * (SL > SU ? 10 : 13) < best * 18) {
            if (sbt_status st = sbt_cuda_check(sbt_launch_dependent(line, dim3((unsigned)std::min<int64_t>(p.items, blocks)),
                                                                    dim3(32 * L::WARPS), L::SMEM, stream, p),
                                               "matvec_e2m1 launch"))
                return st;
            return sbt_after_launch(ctx, "matvec_e2m1");
        }
    }
    if (sbt_status st = sbt_cuda_check(
            sbt_launch_dependent_cluster(kern, dim3((unsigned)(tiles * p.ranks), (unsigned)chunks), dim3(32 * S::WARPS),
                                         (unsigned)p.ranks, S::SMEM, stream, p),
            "matvec_e2m1 launch"))
        return st;
    return sbt_after_launch(ctx, "matvec_e2m1");
}

template <int KIND, int U, bool E4M3, int MT>
sbt_status pick_stage(sbt_context* ctx, MatvecParams& p, cudaStream_t stream) {
    const bool aligned = sbt_aligned16(p.w) && p.ld_w % 16 == 0;
    // (neither fp32 nor 16 rows beside eleven other warps leave registers for 64 k of x)
    constexpr int FEW = MT == 1 ? 64 / U : 1;
    if constexpr (KIND != kF32)
        if (p.K % 64 == 0 && (p.group % 64 == 0 || 64 % p.group == 0) && aligned)
            return launch<KIND, U, FEW, 64 / U, E4M3, MT, true>(ctx, p, stream);
    return aligned ? launch<KIND, U, 1, 1, E4M3, MT, true>(ctx, p, stream) : launch<KIND, U, 1, 1, E4M3, MT, false>(ctx, p, stream);
}

template <int KIND, bool E4M3>
sbt_status pick(sbt_context* ctx, MatvecParams& p, cudaStream_t stream) {
    const bool wide = p.group % 32 == 0, two = p.tokens > 8;
    p.x_vec = ((uintptr_t)p.x | (uintptr_t)p.ld_x) % (KIND != kF32 && !wide ? 8 : 16) == 0;
    if (wide) return two ? pick_stage<KIND, 32, E4M3, 2>(ctx, p, stream) : pick_stage<KIND, 32, E4M3, 1>(ctx, p, stream);
    return two ? pick_stage<KIND, 16, E4M3, 2>(ctx, p, stream) : pick_stage<KIND, 16, E4M3, 1>(ctx, p, stream);
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
        case kF32: return e4m3_scales ? pick<kF32, true>(ctx, p, stream) : pick<kF32, false>(ctx, p, stream);
        case kBF16: return e4m3_scales ? pick<kBF16, true>(ctx, p, stream) : pick<kBF16, false>(ctx, p, stream);
        default: return e4m3_scales ? pick<kF16, true>(ctx, p, stream) : pick<kF16, false>(ctx, p, stream);
    }
}
