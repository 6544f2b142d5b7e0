// What a step's operators read about its new tokens, built on the device from
// the requests' lengths: prefix sums, and each token's sequence, position and
// slot; and for trees of drafted tokens their masks and positions.
//
// Integers only, a few bytes a token, so a call costs what its launch and its
// chain of dependent loads cost.  One launch does everything: every block sums
// all counts for itself (a pass over 65,536 counts is 256 KB from L2), which is
// less than a second launch, and finds the owners of its own tokens in shared
// memory: an entry marks its first token of the block, and a running maximum
// over the marks gives every token its entry, whatever the counts are.  Measured
// (GB300): a token each of 256 entries 5.3 us, what the host takes for a call (3.3 in
// a graph); the slots of prompts 5.8, in a graph too.
#include <algorithm>

#include "sbt_internal.cuh"
#include "tc_ptx.cuh"

namespace {

using sbt_ptx::griddep_wait;

constexpr int kThreads = 256;
constexpr int kTokens = 1024;  // tokens of a block, and entries of a step of the prefix sum

struct SlotParams {
    const int32_t *n_new, *seqs, *start, *lens, *table;  // seqs, start may be NULL
    int32_t *cu, *seq, *positions, *slots, *last;        // each may be NULL
    int64_t ld_table, n_pages;
    int32_t batch, capacity, n_seq, max_pages;
    sbt_fastdiv page_size;
};

// Inclusive scan of one value per thread over the block; every thread gets its prefix.
template <typename T, class F>
__device__ __forceinline__ T block_scan(T v, T* s_warp, F op) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v = op(v, y);
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v = op(v, s_warp[w]);
    return v;
}

__global__ void __launch_bounds__(kThreads) k_pages_slots(const SlotParams p) {
    constexpr int PER = kTokens / kThreads;
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ int32_t s_max[kThreads / 32];
    __shared__ int64_t s_total;
    __shared__ int32_t s_entry[kTokens], s_begin[kTokens], s_mark[kTokens];  // of the entry that begins here; the last mark
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * kTokens, t1 = t0 + kTokens;
    for (int i = threadIdx.x; i < kTokens; i += kThreads) s_entry[i] = -1;
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.cu) p.cu[0] = 0;
    __syncthreads();

    int64_t before = 0;
    uint32_t writer = 0;  // the block that writes this step's entries
    for (int64_t e0 = 0; e0 < p.batch; e0 += kTokens) {
        int32_t n[PER];
        int64_t mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t e = e0 + threadIdx.x * PER + i;
            n[i] = e < p.batch ? max(sbt_ld(p.n_new + e), 0) : 0;
            mine += n[i];
        }
        const int64_t up_to = block_scan<int64_t>(mine, s_sum, [](int64_t a, int64_t b) { return a + b; });
        if (threadIdx.x == kThreads - 1) s_total = up_to;
        int64_t at = before + up_to - mine;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t e = e0 + threadIdx.x * PER + i, end = at + n[i];
            if (n[i] > 0 && at < t1 && end > t0) {
                const int m = (int)(max(at, t0) - t0);
                s_entry[m] = (int32_t)e, s_begin[m] = (int32_t)at;
            }
            if (writer == blockIdx.x && e < p.batch) {
                if (p.cu) p.cu[e + 1] = (int32_t)min(end, (int64_t)p.capacity);
                if (p.last) p.last[e] = n[i] > 0 && end <= p.capacity ? (int32_t)(end - 1) : -1;
            }
            at = end;
        }
        __syncthreads();
        before += s_total;
        if (++writer == gridDim.x) writer = 0;
    }

    int32_t mark = -1, marks[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (s_entry[threadIdx.x * PER + i] >= 0) mark = threadIdx.x * PER + i;
        marks[i] = mark;
    }
    const int32_t top = block_scan<int32_t>(mark, s_max, [](int32_t a, int32_t b) { return max(a, b); });
    const int32_t left = __shfl_up_sync(0xffffffffu, top, 1);
    int32_t prior = (threadIdx.x & 31) ? left : -1;
    for (int w = 0; w < (int)(threadIdx.x >> 5); ++w) prior = max(prior, s_max[w]);
#pragma unroll
    for (int i = 0; i < PER; ++i) s_mark[threadIdx.x * PER + i] = max(marks[i], prior);
    __syncthreads();

#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int k = i * kThreads + threadIdx.x;
        const int64_t t = t0 + k;
        if (t >= p.capacity) break;
        int32_t seq = -1, position = -1, slot = -1;
        const int32_t m = s_mark[k];
        if (t < before && m >= 0) {
            const int32_t e = s_entry[m], begin = s_begin[m], s = p.seqs ? sbt_ld(p.seqs + e) : e;
            if (s >= 0 && s < p.n_seq) {
                seq = s;
                int64_t first;
                if (p.start) {
                    first = sbt_ld(p.start + e);
                } else {
                    const int64_t room = (int64_t)p.max_pages * p.page_size.d, len = sbt_ld(p.lens + s);
                    first = min(max(len, (int64_t)0), room) - max(sbt_ld(p.n_new + e), 0);
                }
                const int64_t at = first + (t - begin);
                if (at >= 0 && at < (1ll << 31)) {
                    position = (int32_t)at;
                    const uint32_t j = sbt_div(p.page_size, (uint32_t)position);
                    if (p.slots && j < (uint32_t)p.max_pages) {
                        const int32_t page = sbt_ld(p.table + (int64_t)s * p.ld_table + j);
                        if (page >= 0 && page < p.n_pages)
                            slot = (int32_t)((int64_t)page * p.page_size.d + (position - (int64_t)j * p.page_size.d));
                    }
                }
            }
        }
        if (p.seq) p.seq[t] = seq;
        if (p.positions) p.positions[t] = position;
        if (p.slots) p.slots[t] = slot;
    }
}

struct TreeParams {
    const int32_t *parents, *cu, *positions;
    int32_t *turned;
    uint32_t* mask;
    int64_t ld_mask;
    int32_t batch, rows, words;
};

// A thread per token: its entry by bisection, then up its chain of parents,
// whose numbers only fall, so the mask's words are finished one after another
// from the token's own down.
__global__ void __launch_bounds__(kThreads) k_tree_plan(const TreeParams p) {
    griddep_wait();
    const int64_t row = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (row >= p.rows) return;
    int32_t lo = 0, hi = p.batch;  // the last entry that begins at or before the row
    while (lo < hi) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (sbt_ld(p.cu + mid + 1) <= row) lo = mid + 1; else hi = mid;
    }
    uint32_t* const mask = p.mask ? p.mask + row * p.ld_mask : nullptr;
    const int32_t begin = lo < p.batch ? sbt_ld(p.cu + lo) : 0;
    if (lo >= p.batch || begin < 0 || begin > row) {  // no entry's token
        for (int w = 0; mask && w < p.words; ++w) mask[w] = 0;
        if (p.turned) p.turned[row] = -1;
        return;
    }
    const int32_t i = (int32_t)row - begin;
    int32_t j = i, depth = 0, w = p.words;
    uint32_t bits = 0;
    while (true) {
        if (mask) {
            for (; w > (j >> 5); --w, bits = 0)  // the word of the tokens walked so far is done, those below hold nothing yet
                if (w < p.words) mask[w] = bits;
            if ((j >> 5) < p.words) bits |= 1u << (j & 31);
        }
        const int32_t up = sbt_ld(p.parents + begin + j);
        if (up < 0 || up >= j) break;
        j = up, ++depth;
    }
    if (mask)
        for (; w >= 0; --w, bits = 0)
            if (w < p.words) mask[w] = bits;
    if (p.turned) {
        const int32_t at = sbt_ld(p.positions + row);
        p.turned[row] = at < 0 ? -1 : at - i + depth;
    }
}

}  // namespace

sbt_status sbt_launch_pages_slots(sbt_context* ctx, const sbt_page_map* m, const int32_t* n_new, int32_t batch,
                                  const int32_t* seqs, const int32_t* start, int32_t capacity, int32_t* cu,
                                  int32_t* seq, int32_t* positions, int32_t* slots, int32_t* last,
                                  cudaStream_t stream) {
    SlotParams p = {};
    p.n_new = n_new, p.seqs = seqs, p.start = start, p.lens = m->lens, p.table = m->page_table;
    p.cu = cu, p.seq = seq, p.positions = positions, p.slots = slots, p.last = last;
    p.ld_table = m->ld_table, p.n_pages = m->n_pages;
    p.batch = batch, p.capacity = capacity, p.n_seq = m->n_seq, p.max_pages = m->max_pages;
    p.page_size = sbt_make_fastdiv((uint32_t)m->page_size);
    const bool tokens = seq || positions || slots;
    const int64_t blocks = std::max<int64_t>(1, tokens ? sbt_cdiv(capacity, kTokens) : 1);
    if (sbt_status st = sbt_cuda_check(sbt_launch_dependent(k_pages_slots, dim3((unsigned)blocks), dim3(kThreads), 0,
                                                            stream, p),
                                       "pages_slots launch"))
        return st;
    return sbt_after_launch(ctx, "pages_slots");
}

sbt_status sbt_launch_tree_plan(sbt_context* ctx, const int32_t* parents, const int32_t* cu, int32_t batch,
                                int32_t rows, const int32_t* positions, int32_t* turned, int32_t* mask,
                                int64_t ld_mask, cudaStream_t stream) {
    TreeParams p = {};
    p.parents = parents, p.cu = cu, p.positions = positions, p.turned = turned;
    p.mask = (uint32_t*)mask, p.ld_mask = ld_mask, p.words = (int32_t)ld_mask;
    p.batch = batch, p.rows = rows;
    if (sbt_status st = sbt_cuda_check(sbt_launch_dependent(k_tree_plan, dim3((unsigned)sbt_cdiv(rows, kThreads)),
                                                            dim3(kThreads), 0, stream, p),
                                       "tree_plan launch"))
        return st;
    return sbt_after_launch(ctx, "tree_plan");
}
