// Pages of a cache: copy, reserve (grow), fork, free (cut) and compact.
//
// The state is the caller's: a table of page numbers per sequence, the
// sequences' lengths, and a count of holders per page (0: free).  Every
// decision is taken on the device from that state, and every result is a
// function of it alone: free pages are given lowest number first, requests are
// served in order, and the counts change by integer atomics whose order cannot
// be seen.
//
// Extents go up to 2^31 - 1, so counters that step past one have 64 bits.
//
// Deciding is a few prefix sums over the sequences and the pages; one block of
// 1024 threads does it (a pass over 65,536 counts is 256 KB) and leaves a plan
// in the workspace.  Moving the pages' bytes is memory-bound; the second
// kernel spreads the plan's rows and pages over the GPU.
#include <algorithm>

#include "sbt_internal.cuh"
#include "tc_ptx.cuh"

namespace {

using sbt_ptx::griddep_wait;

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 4;                                    // 16-byte vectors per thread and chunk
constexpr int kMoveBlocks = 32;                                 // blocks per SM at most (8: 173 us, 32: 159 us for 1 GB each way)
constexpr int kChunkBytes = kMoveThreads * kMoveVecs * 16;

struct Pool {
    char* base;
    int64_t plane_stride, page_stride, page_bytes;
    int32_t planes, chunks;  // chunks of one page
};

struct Pools {
    Pool p[SBT_MAX_PAGE_POOLS];
    int32_t n;
    int32_t width;           // 16, 4 or 1: every address and size is a multiple of it
    int64_t chunks;          // chunks of one page number: over all pools and planes
};

struct Map {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    int64_t ld;
    int32_t n_seq, max_pages, n_pages;
    sbt_fastdiv page_size;
    __device__ __forceinline__ int32_t pages_of(int32_t len) const {
        return len <= 0 ? 0 : (int32_t)sbt_div(page_size, (uint32_t)(len - 1)) + 1;
    }
    __device__ __forceinline__ int32_t held(int32_t len) const { return min(pages_of(len), max_pages); }
    __device__ __forceinline__ bool page_ok(int32_t p) const { return p >= 0 && p < n_pages; }
};

// Workspace: counts, then the lists.
struct Plan {
    int32_t* count;   // [0]: page moves
    int32_t* src;     // page moves
    int32_t* dst;
    int32_t* free;    // free pages, ascending
    int32_t* claim;   // fork: lowest pair that wants this child
    int32_t* a;       // per sequence or pair
    int32_t* b;
    int32_t* c;
};

size_t plan_bytes(int32_t n_seq, int64_t n_pages) {
    const int64_t moves = std::max<int64_t>(n_pages, n_seq);
    return 256 + 4 * (size_t)(2 * moves + n_pages + 4 * (int64_t)n_seq);
}

Plan plan_of(void* ws, int32_t n_seq, int64_t n_pages) {
    const int64_t moves = std::max<int64_t>(n_pages, n_seq);
    Plan w;
    w.count = (int32_t*)ws;
    w.src = w.count + 64;
    w.dst = w.src + moves;
    w.free = w.dst + moves;
    w.claim = w.free + n_pages;
    w.a = w.claim + n_seq;
    w.b = w.a + n_seq;
    w.c = w.b + n_seq;
    return w;
}

// Exclusive prefix of one value per thread over the block, and the block's sum.
template <typename T>
__device__ __forceinline__ T scan(T v, T* total, T* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    T w = s_warp[lane], t = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, t, d);
        if (lane >= d) t += y;
    }
    *total = __shfl_sync(0xffffffffu, t, 31);
    return __shfl_sync(0xffffffffu, t - w, warp) + x - v;
}

// The first pages whose count is 0, ascending, into `list` (at least `want` of
// them if there are as many); returns how many were found.
__device__ int32_t collect_free(const Map& m, int32_t want, int32_t* list, int32_t* s_warp) {
    int32_t found = 0;
    for (int64_t p0 = 0; p0 < m.n_pages && found < want; p0 += 4 * kPlanThreads) {
        const int64_t p = p0 + 4 * threadIdx.x;
        bool f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = p + i < m.n_pages && m.refs[p + i] <= 0;
        int32_t total, at = found + scan<int32_t>(f[0] + f[1] + f[2] + f[3], &total, s_warp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (f[i]) list[at++] = (int32_t)(p + i);
        found += total;
    }
    return found;
}

// ------------------------------------------------------------------------------ page bytes

// Chunk `r` of the page number pair (src, dst).
__device__ __forceinline__ void move_chunk(const Pools& q, int64_t r, int32_t src, int32_t dst) {
    int k = 0;
    while (k + 1 < q.n && r >= (int64_t)q.p[k].planes * q.p[k].chunks) {
        r -= (int64_t)q.p[k].planes * q.p[k].chunks;
        ++k;
    }
    const Pool& o = q.p[k];
    const int64_t plane = r / o.chunks, at = (r - plane * o.chunks) * kChunkBytes;
    const char* s = o.base + plane * o.plane_stride + src * o.page_stride + at;
    char* d = o.base + plane * o.plane_stride + dst * o.page_stride + at;
    const int64_t left = o.page_bytes - at;
    const int n = left < kChunkBytes ? (int)left : kChunkBytes;
    if (q.width == 16) {
        uint4 v[kMoveVecs];
#pragma unroll
        for (int i = 0; i < kMoveVecs; ++i) {
            const int b = (i * kMoveThreads + threadIdx.x) * 16;
            if (b < n) v[i] = *reinterpret_cast<const uint4*>(s + b);
        }
#pragma unroll
        for (int i = 0; i < kMoveVecs; ++i) {
            const int b = (i * kMoveThreads + threadIdx.x) * 16;
            if (b < n) sbt_st_v4_cs(d + b, v[i]);
        }
    } else if (q.width == 4) {
#pragma unroll 8
        for (int b = threadIdx.x * 4; b < n; b += kMoveThreads * 4)
            *reinterpret_cast<uint32_t*>(d + b) = *reinterpret_cast<const uint32_t*>(s + b);
    } else {
#pragma unroll 8
        for (int b = threadIdx.x; b < n; b += kMoveThreads) d[b] = s[b];
    }
}

__device__ __forceinline__ void move_pages(const Pools& q, const int32_t* src, const int32_t* dst, int64_t n,
                                           int32_t n_pages) {
    const int64_t jobs = n * q.chunks;
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int64_t i = job / q.chunks;
        const int32_t s = sbt_ld(src + i), d = sbt_ld(dst + i);
        if (s < 0 || s >= n_pages || d < 0 || d >= n_pages || s == d) continue;
        move_chunk(q, job - i * q.chunks, s, d);
    }
}

__global__ void __launch_bounds__(kMoveThreads) k_pages_copy(const __grid_constant__ Pools q, const int32_t* src,
                                                             const int32_t* dst, int64_t n, int32_t n_pages) {
    griddep_wait();
    move_pages(q, src, dst, n, n_pages);
}

// The moves of a plan (their number is on the device).
__global__ void __launch_bounds__(kMoveThreads) k_pages_moves(const __grid_constant__ Pools q, const Plan w,
                                                              int32_t n_pages) {
    griddep_wait();
    move_pages(q, w.src, w.dst, *w.count, n_pages);
}

// ------------------------------------------------------------------------------------ free

__global__ void __launch_bounds__(kMoveThreads) k_pages_free(const Map m, const int32_t* seqs, const int32_t* keep) {
    griddep_wait();
    const int32_t s = sbt_ld(seqs + blockIdx.x);
    if (s < 0 || s >= m.n_seq) return;
    int32_t k = keep ? sbt_ld(keep + blockIdx.x) : 0;
    if (k < 0) k = 0;
    // a sequence listed twice: both occurrences may see the old length; the exchange lets only one of
    // them release a page
    const int32_t end = m.held(*(volatile int32_t*)(m.lens + s));
    for (int64_t j = (int64_t)m.pages_of(k) + threadIdx.x; j < end; j += kMoveThreads) {
        const int32_t p = atomicExch(m.table + s * m.ld + j, -1);
        if (m.page_ok(p)) atomicSub(m.refs + p, 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) atomicMin(m.lens + s, k);
}

// --------------------------------------------------------------------------------- reserve

__global__ void __launch_bounds__(kPlanThreads) k_pages_reserve(const Map m, const Plan w, const int32_t* target) {
    griddep_wait();
    __shared__ int32_t s_warp[32];
    __shared__ int64_t s_warp64[32];
    __shared__ int32_t s_moves;
    if (threadIdx.x == 0) s_moves = 0;
    // need[b]: pages past the ones held, and one more where the last page is part full and shared.  What all
    // sequences ask for may add up to n_seq * max_pages, far more than any pool holds: 64 bits.
    int64_t total = 0;
    for (int64_t b0 = 0; b0 < m.n_seq; b0 += kPlanThreads) {
        const int64_t b = b0 + threadIdx.x;
        int32_t need = 0, own = 0;
        if (b < m.n_seq) {
            const int32_t n = max(m.lens[b], 0), t = sbt_ld(target + b);
            if (t > n && m.pages_of(t) <= m.max_pages) {
                need = m.pages_of(t) - m.pages_of(n);
                if (n > 0 && n - (int32_t)(sbt_div(m.page_size, (uint32_t)n) * m.page_size.d) != 0) {
                    const int32_t p = m.table[b * m.ld + m.pages_of(n) - 1];
                    own = m.page_ok(p) && m.refs[p] > 1;
                }
                need += own;
            }
            w.a[b] = need;
            w.b[b] = own;
        }
        int64_t sum;
        const int64_t at = total + scan<int64_t>(need, &sum, s_warp64);
        if (b < m.n_seq) w.c[b] = (int32_t)min(at, (int64_t)INT32_MAX);  // there: past every list
        total += sum;
    }
    const int32_t found = total ? collect_free(m, (int32_t)min(total, (int64_t)m.n_pages), w.free, s_warp) : 0;
    __syncthreads();
    // a warp per sequence: served if it needs no page or its pages end inside the list
    for (int64_t b = threadIdx.x >> 5; b < m.n_seq; b += kPlanThreads / 32) {
        const int lane = threadIdx.x & 31;
        const int32_t n = max(m.lens[b], 0), t = sbt_ld(target + b), need = w.a[b], own = w.b[b], at = w.c[b];
        if (t <= n || m.pages_of(t) > m.max_pages || (need && need > found - at)) continue;
        const int32_t first = m.pages_of(n) - own;
        for (int64_t i = lane; i < need; i += 32) {
            const int32_t p = w.free[at + i];
            if (i == 0 && own) {
                const int32_t old = m.table[b * m.ld + first];
                const int32_t k = atomicAdd(&s_moves, 1);
                w.src[k] = old;
                w.dst[k] = p;
                atomicSub(m.refs + old, 1);
            }
            m.table[b * m.ld + first + i] = p;
            m.refs[p] = 1;
        }
        __syncwarp();
        if (lane == 0) m.lens[b] = t;
    }
    __syncthreads();
    if (threadIdx.x == 0) *w.count = s_moves;
}

// ------------------------------------------------------------------------------------ fork

__global__ void __launch_bounds__(kPlanThreads) k_pages_fork(const Map m, const Plan w, const int32_t* from,
                                                             const int32_t* to, int32_t n) {
    griddep_wait();
    __shared__ int32_t s_warp[32];
    auto ok = [&](int64_t i, int32_t& a, int32_t& c) {
        a = sbt_ld(from + i), c = sbt_ld(to + i);
        return a >= 0 && a < m.n_seq && c >= 0 && c < m.n_seq && a != c && m.lens[a] > 0 && m.lens[c] <= 0;
    };
    int32_t a, c;
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads)
        if (ok(i, a, c)) w.claim[c] = 0x7fffffff;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads)
        if (ok(i, a, c)) atomicMin(w.claim + c, (int32_t)i);
    __syncthreads();
    // a[i]: parent's length or 0 (pair not taken); b[i]: place of the child's last page in the free list or -1
    int32_t total = 0;
    for (int64_t i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int64_t i = i0 + threadIdx.x;
        int32_t len = 0, part = 0;
        if (i < n && ok(i, a, c) && w.claim[c] == i) {
            len = m.lens[a];
            if (len - (int32_t)(sbt_div(m.page_size, (uint32_t)len) * m.page_size.d) != 0 &&
                m.pages_of(len) <= m.max_pages)
                part = m.page_ok(m.table[a * m.ld + m.pages_of(len) - 1]);
        }
        int32_t sum;
        const int32_t at = total + scan(part, &sum, s_warp);
        if (i < n) {
            w.a[i] = len;
            w.b[i] = part ? at : -1;
        }
        total += sum;
    }
    const int32_t found = total ? collect_free(m, total, w.free, s_warp) : 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t len = w.a[i], at = w.b[i];
        int32_t src = -1, dst = -1;
        if (len > 0) {
            a = sbt_ld(from + i), c = sbt_ld(to + i);
            if (at >= found) {
                w.a[i] = 0;  // no page left for its last tokens: not taken
            } else {
                if (at >= 0) {
                    src = m.table[a * m.ld + m.pages_of(len) - 1];
                    dst = w.free[at];
                    m.refs[dst] = 1;
                }
                m.lens[c] = len;
            }
        }
        w.src[i] = src;
        w.dst[i] = dst;
    }
    if (threadIdx.x == 0) *w.count = n;
}

// The children's rows (block per pair), then the copies of the last pages.
__global__ void __launch_bounds__(kMoveThreads) k_pages_fork_rows(const __grid_constant__ Pools q, const Map m,
                                                                  const Plan w, const int32_t* from, const int32_t* to,
                                                                  int32_t n) {
    griddep_wait();
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const int32_t len = w.a[i];
        if (len <= 0) continue;
        const int32_t a = sbt_ld(from + i), c = sbt_ld(to + i), pages = m.held(len);
        for (int64_t j = threadIdx.x; j < pages; j += kMoveThreads) {
            int32_t p = m.table[a * m.ld + j];
            if (j == pages - 1 && w.dst[i] >= 0) {
                p = w.dst[i];
            } else if (m.page_ok(p)) {
                atomicAdd(m.refs + p, 1);
            }
            m.table[c * m.ld + j] = p;
        }
    }
    move_pages(q, w.src, w.dst, n, m.n_pages);
}

// --------------------------------------------------------------------------------- compact

struct Packed {
    int32_t* table;   // may be the map's own
    int64_t ld;
    int32_t* refs;    // may be the map's own
    int32_t* page_to;
    int32_t* n_live;
};

// With L live pages, the live ones at L and above move, in order, into the
// holes below L: the fewest moves that pack the pool, and no page is both read
// and written.
__global__ void __launch_bounds__(kPlanThreads) k_pages_compact(const Map m, const Plan w, const Packed o) {
    griddep_wait();
    __shared__ int32_t s_warp[32];
    int32_t mine = 0, live;
    for (int64_t p = threadIdx.x; p < m.n_pages; p += kPlanThreads) mine += m.refs[p] > 0;
    scan(mine, &live, s_warp);
    int32_t holes = 0, movers = 0;
    for (int64_t p0 = 0; p0 < m.n_pages; p0 += kPlanThreads) {
        const int64_t p = p0 + threadIdx.x;
        const bool in = p < m.n_pages, used = in && m.refs[p] > 0;
        const bool hole = in && !used && p < live, mover = used && p >= live;
        // both prefixes in one scan: at most kPlanThreads of each
        int32_t sum;
        const int32_t at = scan(mover ? 1 << 16 : hole ? 1 : 0, &sum, s_warp);
        if (hole) w.dst[holes + (at & 0xFFFF)] = (int32_t)p;
        if (mover) w.src[movers + (at >> 16)] = (int32_t)p;
        // until the holes are known a mover's place holds -2 - its rank
        if (in) o.page_to[p] = mover ? -2 - (movers + (at >> 16)) : used ? (int32_t)p : -1;
        holes += sum & 0xFFFF;
        movers += sum >> 16;
    }
    __syncthreads();
    for (int64_t p = threadIdx.x; p < m.n_pages; p += kPlanThreads) {
        const int32_t to = o.page_to[p];
        if (to >= 0) {
            o.refs[p] = m.refs[p];
        } else if (to <= -2) {
            const int32_t d = w.dst[-2 - to];
            o.page_to[p] = d;
            o.refs[d] = m.refs[p];
            o.refs[p] = 0;
        } else if (p >= live) {
            o.refs[p] = 0;
        }
    }
    if (threadIdx.x == 0) {
        *w.count = movers;
        *o.n_live = live;
    }
}

__global__ void __launch_bounds__(kMoveThreads) k_pages_compact_rows(const __grid_constant__ Pools q, const Map m,
                                                                     const Plan w, const Packed o) {
    griddep_wait();
    for (int64_t s = blockIdx.x; s < m.n_seq; s += gridDim.x) {
        const int32_t pages = m.held(m.lens[s]);
        for (int64_t j = threadIdx.x; j < pages; j += kMoveThreads) {
            const int32_t p = m.table[s * m.ld + j];
            o.table[s * o.ld + j] = m.page_ok(p) ? o.page_to[p] : -1;
        }
    }
    move_pages(q, w.src, w.dst, *w.count, m.n_pages);
}

// ------------------------------------------------------------------------------------ host

Map map_of(const sbt_page_map* map) {
    Map m;
    m.table = map->page_table, m.lens = map->lens, m.refs = map->refs;
    m.ld = map->ld_table, m.n_seq = map->n_seq, m.max_pages = map->max_pages, m.n_pages = (int32_t)map->n_pages;
    m.page_size = sbt_make_fastdiv((uint32_t)map->page_size);
    return m;
}

Pools pools_of(const sbt_page_pool* pools, int32_t n) {
    Pools q = {};
    q.n = n;
    uint64_t bits = 16;
    for (int i = 0; i < n; ++i) {
        const sbt_page_pool& s = pools[i];
        Pool& d = q.p[i];
        d.base = (char*)s.base, d.plane_stride = s.plane_stride, d.page_stride = s.page_stride;
        d.page_bytes = s.page_bytes, d.planes = (int32_t)s.n_planes;
        d.chunks = (int32_t)sbt_cdiv(s.page_bytes, kChunkBytes);
        q.chunks += s.n_planes * d.chunks;
        bits |= reinterpret_cast<uintptr_t>(s.base) | (uint64_t)(s.plane_stride | s.page_stride | s.page_bytes);
    }
    q.width = bits & 3 ? 1 : bits & 15 ? 4 : 16;
    return q;
}

// Every launch is a programmatic dependent: the kernels wait for the one ahead before they touch memory.
sbt_status launched(sbt_context* ctx, const char* what, cudaError_t e) {
    const sbt_status st = sbt_cuda_check(e, what);
    return st ? st : sbt_after_launch(ctx, what);
}

int move_grid(const sbt_context* ctx, int64_t jobs) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(jobs, (int64_t)ctx->sm_count * kMoveBlocks));
}

}  // namespace

size_t sbt_pages_workspace_bytes(int32_t n_seq, int64_t n_pages) { return plan_bytes(n_seq, n_pages); }

sbt_status sbt_launch_pages_copy(sbt_context* ctx, const sbt_page_pool* pools, int32_t n_pools, int64_t n_pages,
                                 const int32_t* src, const int32_t* dst, int64_t n, cudaStream_t stream) {
    const Pools q = pools_of(pools, n_pools);
    return launched(ctx, "pages_copy",
                    sbt_launch_dependent(k_pages_copy, dim3(move_grid(ctx, n * q.chunks)), dim3(kMoveThreads), 0,
                                         stream, q, src, dst, n, (int32_t)n_pages));
}

sbt_status sbt_launch_pages_free(sbt_context* ctx, const sbt_page_map* map, const int32_t* seqs, const int32_t* keep,
                                 int32_t n, cudaStream_t stream) {
    return launched(ctx, "pages_free",
                    sbt_launch_dependent(k_pages_free, dim3(n), dim3(kMoveThreads), 0, stream, map_of(map), seqs, keep));
}

sbt_status sbt_launch_pages_reserve(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools,
                                    int32_t n_pools, const int32_t* target, void* workspace, cudaStream_t stream) {
    const Map m = map_of(map);
    const Plan w = plan_of(workspace, map->n_seq, map->n_pages);
    const Pools q = pools_of(pools, n_pools);
    const sbt_status st = launched(ctx, "pages_reserve", sbt_launch_dependent(k_pages_reserve, dim3(1), dim3(kPlanThreads),
                                                                              0, stream, m, w, target));
    if (st) return st;
    return launched(ctx, "pages_reserve moves",
                    sbt_launch_dependent(k_pages_moves, dim3(move_grid(ctx, map->n_seq * q.chunks)),
                                         dim3(kMoveThreads), 0, stream, q, w, m.n_pages));
}

sbt_status sbt_launch_pages_fork(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools,
                                 int32_t n_pools, const int32_t* from, const int32_t* to, int32_t n, void* workspace,
                                 cudaStream_t stream) {
    const Map m = map_of(map);
    const Plan w = plan_of(workspace, map->n_seq, map->n_pages);
    const Pools q = pools_of(pools, n_pools);
    const sbt_status st = launched(ctx, "pages_fork", sbt_launch_dependent(k_pages_fork, dim3(1), dim3(kPlanThreads), 0,
                                                                           stream, m, w, from, to, n));
    if (st) return st;
    return launched(ctx, "pages_fork rows",
                    sbt_launch_dependent(k_pages_fork_rows, dim3(move_grid(ctx, n * q.chunks)), dim3(kMoveThreads), 0,
                                         stream, q, m, w, from, to, n));
}

sbt_status sbt_launch_pages_compact(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools,
                                    int32_t n_pools, int32_t* table_out, int64_t ld_out, int32_t* refs_out,
                                    int32_t* page_to, int32_t* n_live, void* workspace, cudaStream_t stream) {
    const Map m = map_of(map);
    const Plan w = plan_of(workspace, map->n_seq, map->n_pages);
    const Pools q = pools_of(pools, n_pools);
    const Packed o = {table_out, ld_out, refs_out, page_to, n_live};
    const sbt_status st = launched(ctx, "pages_compact", sbt_launch_dependent(k_pages_compact, dim3(1), dim3(kPlanThreads),
                                                                              0, stream, m, w, o));
    if (st) return st;
    const int64_t jobs = std::max<int64_t>(map->n_seq, (map->n_pages / 2) * q.chunks);
    return launched(ctx, "pages_compact rows",
                    sbt_launch_dependent(k_pages_compact_rows, dim3(move_grid(ctx, jobs)), dim3(kMoveThreads), 0,
                                         stream, q, m, w, o));
}
