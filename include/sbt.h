/*
 * sbt.h -- bounds-checked tile movement, a boundary-tile bf16 GEMM, the
 * operators of a paged key-value cache and those between a layer's GEMMs on one
 * NVIDIA GB300 (sm_103a).  C ABI of libsbt.so.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Coordinates are zero-based and signed 64-bit; negative origins are legal
 *    (Tylo.jl "Boundary tiles": the origin and all coordinates are zero-based,
 *    negative crop origins are supported).
 *  - Arrays are row-major with explicit strides counted in ELEMENTS.  A
 *    column-major array is the same call with the strides swapped.
 *  - Movement calls copy raw element bits (dtype only fixes the element size);
 *    NaN payloads and -0.0 are preserved bit for bit.
 *  - All array pointers are DEVICE pointers (cudaMalloc'd or otherwise
 *    device-addressable).  `pad_value` is a HOST pointer to one element's bits.
 *    The caller owns every buffer; the library allocates no device memory.
 *  - Every array pointer is a multiple of its element size (int32 indices and
 *    cu_seqlens: 4 bytes; 8-bit codes, scales and masks: any address); a call
 *    given one that is not returns SBT_ERR_ALIGNMENT before any launch.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream) and returns after enqueueing.  Arguments are validated on
 *    the host before anything is launched; on error nothing is launched and
 *    sbt_last_error_message() says why.  A call whose output is empty returns
 *    SBT_OK without launching.
 *  - Metadata that lives on the device (indices, cu_seqlens) cannot be checked
 *    on the host: out-of-range values are handled by the semantics (pad on
 *    load, clip on store), never by faulting.
 *  - Kernels that wait on hardware barriers bound every wait; a wait that runs
 *    out sets a per-device status flag, the kernel returns early and
 *    sbt_check_status() reports SBT_ERR_DEVICE_TIMEOUT.
 */
#ifndef SBT_H_
#define SBT_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SBT_API __attribute__((visibility("default")))
#else
#define SBT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SBT_OK = 0,
    SBT_ERR_INVALID_ARG = 1,    /* null pointer, negative extent, bad stride, tile too large, ... */
    SBT_ERR_UNSUPPORTED = 2,    /* dtype or combination this op does not take */
    SBT_ERR_ALIGNMENT = 3,      /* array pointer not on a multiple of its element size; workspace not
                                   256-byte aligned or too small */
    SBT_ERR_TENSOR_MAP = 4,     /* the driver refused a TMA descriptor (Mojo "RaggedTMA3DTile": create raises) */
    SBT_ERR_CUDA = 5,           /* a CUDA runtime/driver call failed */
    SBT_ERR_DEVICE_TIMEOUT = 6  /* a bounded device-side wait ran out (see sbt_check_status) */
} sbt_status;

typedef enum { SBT_F32 = 0, SBT_BF16 = 1, SBT_F16 = 2 } sbt_dtype;

/* Which copy path the host may pick.  AUTO chooses per call from alignment:
 * TMA for aligned interior tiles, 16-byte vectors where the addresses allow,
 * scalar bounds-checked elements otherwise.  The others force one path where
 * the call allows it (tests and measurements); results are identical.  The
 * clipped store into rows that are not 16-byte aligned (tiles side by side
 * along the row) writes realigned row chunks with TMA bulk copies under AUTO
 * and TMA, and lane-shifted 16-byte stores under VECTOR. */
typedef enum { SBT_PATH_AUTO = 0, SBT_PATH_SCALAR = 1, SBT_PATH_VECTOR = 2, SBT_PATH_TMA = 3 } sbt_path;

typedef struct sbt_context sbt_context;

/* Create a context bound to CUDA device `device` (made current by every call
 * that takes the context).  Host memory only.  Returns SBT_ERR_CUDA if the
 * device cannot be queried, SBT_ERR_UNSUPPORTED if it is not compute 10.3. */
SBT_API sbt_status sbt_create(int device, sbt_context** out);
SBT_API sbt_status sbt_destroy(sbt_context* ctx);

/* Path policy for later calls on this context (default SBT_PATH_AUTO). */
SBT_API sbt_status sbt_set_path(sbt_context* ctx, sbt_path path);
/* Limit of every bounded device-side wait, in nanoseconds (default 2e9). */
SBT_API sbt_status sbt_set_wait_limit_ns(sbt_context* ctx, uint64_t ns);
/* Test hook for the bounded device waits.  SBT_TEST_WITHHOLD_LOAD makes the
 * next GEMM (bf16 or block-scaled tensor path), bulk row and tree attention
 * launches on this context skip their first copy (its signal), so
 * a consumer's bounded wait runs out (no fault, no hang): the kernel sets the
 * status flag, drains and returns, and sbt_check_status() reports
 * SBT_ERR_DEVICE_TIMEOUT.  Stays set until reset with SBT_TEST_NONE. */
typedef enum { SBT_TEST_NONE = 0, SBT_TEST_WITHHOLD_LOAD = 1 } sbt_test_hook;
SBT_API sbt_status sbt_set_test_hook(sbt_context* ctx, sbt_test_hook hook);
/* Number of kernels this context has launched so far. */
SBT_API uint64_t sbt_launch_count(const sbt_context* ctx);
/* Synchronise `stream`, then read and clear the device status flag of the
 * context's device: SBT_ERR_DEVICE_TIMEOUT if a bounded wait ran out since
 * the last check, SBT_ERR_CUDA if the stream reports an error, else SBT_OK. */
SBT_API sbt_status sbt_check_status(sbt_context* ctx, void* stream);
/* Message of the last failing call on this thread ("" if none). */
SBT_API const char* sbt_last_error_message(void);

/*
 * Padded tile load over a grid of tiles.
 * cuTile.jl "Memory", section "Bounds checking" (loads are padded where the
 * tile extends past the array) and section "Tile windows" (tile origins move
 * by a per-dimension step; the host counts tiles with ceiling division).
 *
 *   tile (ti, tj), ti < grid_r, tj < grid_c, starts at
 *     (origin_r + ti*step_r, origin_c + tj*step_c);
 *   dst_tiles[((ti*grid_c + tj)*tile_r + i)*tile_c + j] =
 *     src[r*stride_r + c*stride_c]  if 0 <= r < rows and 0 <= c < cols
 *     *pad_value                    otherwise,
 *   with r = tile origin row + i, c = tile origin column + j.
 *
 * src: device, logical rows x cols with element strides (stride_r, stride_c),
 * both nonzero (negative allowed).  dst_tiles: device, contiguous
 * [grid_r][grid_c][tile_r][tile_c].  1 <= tile_r, tile_c <= 256.
 * pad_value: host pointer to one element of `dtype` (NULL means all-zero bits).
 */
SBT_API sbt_status sbt_tile_load_padded(sbt_context* ctx, sbt_dtype dtype, const void* src, int64_t rows, int64_t cols,
                                int64_t stride_r, int64_t stride_c, int64_t origin_r, int64_t origin_c,
                                int64_t step_r, int64_t step_c, int32_t grid_r, int32_t grid_c, int32_t tile_r,
                                int32_t tile_c, void* dst_tiles, const void* pad_value, void* stream);

/*
 * Clipped tile store: the inverse of sbt_tile_load_padded.
 * cuTile.jl "Memory", section "Bounds checking" (stores are clipped) and
 * Tylo.jl "Boundary tiles", section "Accumulator stores and GEMM" (invalid
 * coordinates are suppressed; memory outside the array is left unchanged).
 * Element (i, j) of tile (ti, tj) is written to dst only when its (r, c) is
 * inside rows x cols; nothing else of dst is touched.  Where windows overlap
 * (step < tile) which write lands is undefined.
 */
SBT_API sbt_status sbt_tile_store_clipped(sbt_context* ctx, sbt_dtype dtype, const void* src_tiles, int32_t grid_r,
                                  int32_t grid_c, int32_t tile_r, int32_t tile_c, void* dst, int64_t rows,
                                  int64_t cols, int64_t stride_r, int64_t stride_c, int64_t origin_r,
                                  int64_t origin_c, int64_t step_r, int64_t step_c, void* stream);

/*
 * Row gather through an int32 index tile.
 * warp.tile_load_indexed, description and "Parameters": element (k, j) reads
 * row row_offset + idx[k] (the offset is added before the check, in 64-bit)
 * and column col_offset + j; every coordinate is checked against both bounds
 * and an element outside reads the padding value, so -1 is a sentinel.
 * cuTile.jl "Memory": an optional per-element mask; masked-out elements read
 * the padding value.
 *
 *   out[k*ld_out + j] = src[(row_offset+idx[k])*ld_src + col_offset + j]
 *                         if mask[k][j] (or no mask) and the coordinate is in
 *                         rows x cols;   *pad_value otherwise,
 *   for k < n_idx, j < tile_c.
 *
 * src: device rows x cols, row stride ld_src >= cols.  idx: device int32[n_idx].
 * mask: device uint8 [n_idx][ld_mask] (nonzero = true) or NULL.  out: device
 * [n_idx][ld_out], ld_out >= tile_c; columns >= tile_c are not written.
 * 1 <= tile_c <= 65536.
 */
SBT_API sbt_status sbt_gather_rows(sbt_context* ctx, sbt_dtype dtype, const void* src, int64_t rows, int64_t cols,
                           int64_t ld_src, const int32_t* idx, int64_t n_idx, int64_t row_offset,
                           int64_t col_offset, int32_t tile_c, const uint8_t* mask, int64_t ld_mask, void* out,
                           int64_t ld_out, const void* pad_value, void* stream);

/*
 * Column gather: the gather along axis 1.
 * warp.tile_load_indexed, description and "Parameters" with axis = 1: element
 * (i, k) reads row row_offset + i and column col_offset + idx[k] (the offset
 * added before the check, in 64-bit); every coordinate is checked against both
 * bounds and an element outside reads the padding value.
 *
 *   out[i*ld_out + k] = src[(row_offset+i)*ld_src + col_offset + idx[k]] or *pad_value,
 *   for i < tile_r, k < n_idx.
 *
 * src: device rows x cols, row stride ld_src >= cols.  idx: device int32[n_idx].
 * out: device [tile_r][ld_out], ld_out >= n_idx.  1 <= tile_r <= 65536.
 */
SBT_API sbt_status sbt_gather_cols(sbt_context* ctx, sbt_dtype dtype, const void* src, int64_t rows, int64_t cols,
                                   int64_t ld_src, const int32_t* idx, int64_t n_idx, int64_t row_offset,
                                   int64_t col_offset, int32_t tile_r, void* out, int64_t ld_out,
                                   const void* pad_value, void* stream);

/*
 * Masked row scatter.
 * cuTile.jl "Memory": scatter writes only where the mask is true and is
 * bounds-checked like every tile memory operation (out-of-range elements are
 * clipped); section "Sparse views": conflicting stores to a repeated index
 * are undefined -- here exactly one of the candidate values lands.
 *
 *   for k < n_idx, j < tile_c: if (mask == NULL or mask[k*ld_mask + j] != 0)
 *   and r = row_offset + idx[k] in [0, rows) and c = col_offset + j in
 *   [0, cols):  dst[r*ld_dst + c] = src[k*ld_src + j].
 *
 * Every other element of dst keeps its bits.
 */
SBT_API sbt_status sbt_scatter_rows_masked(sbt_context* ctx, sbt_dtype dtype, void* dst, int64_t rows, int64_t cols,
                                   int64_t ld_dst, const int32_t* idx, int64_t n_idx, int64_t row_offset,
                                   int64_t col_offset, const void* src, int64_t ld_src, int32_t tile_c,
                                   const uint8_t* mask, int64_t ld_mask, void* stream);

/*
 * Row scatter-add: the adjoint (backward) of sbt_gather_rows.
 * warp.tile_load_indexed, description: in a backward pass the adjoint of the
 * gathered tile is accumulated atomically into the array's gradient at the
 * gathered locations.
 *
 *   for k < n_idx, j < tile_c: if r = row_offset + idx[k] in [0, rows) and
 *   c = col_offset + j in [0, cols):  dst[r*ld_dst + c] += src[k*ld_src + j]
 *
 * Each addition is done in the element type (SBT_F32, SBT_BF16 or SBT_F16)
 * with one rounding to nearest even, by the memory system's atomic add, so
 * repeated indices accumulate; their order is unspecified (results with
 * repeats may differ in the last bits from run to run).  Elements that read
 * padding in the forward pass contribute nothing.  Subnormal fp32 results
 * are outside the contract (the GPU's fp32 atomic add may flush them).
 */
SBT_API sbt_status sbt_scatter_add_rows(sbt_context* ctx, sbt_dtype dtype, void* dst, int64_t rows, int64_t cols,
                                        int64_t ld_dst, const int32_t* idx, int64_t n_idx, int64_t row_offset,
                                        int64_t col_offset, const void* src, int64_t ld_src, int32_t tile_c,
                                        void* stream);

/*
 * Ragged 3D tile load.
 * Mojo "RaggedTMA3DTile", struct description: a packed array
 * [total_rows][heads][depth] whose leading dimension concatenates sequences,
 * read as 2D tiles per head with only the first `dynamic_dim` rows of a tile
 * valid.  Sequence b owns packed rows [cu_seqlens[b], cu_seqlens[b+1]).
 *
 *   out[((b*heads + h)*t_pad + r)*depth + d] =
 *     x[(cu[b]+r)*ld_row + h*ld_head + d]  if r < cu[b+1]-cu[b] and
 *                                            0 <= cu[b]+r < total_rows,
 *     0 (all-zero bits)                    otherwise,
 *   for b < batch, h < heads, r < t_pad, d < depth.
 *
 * x: device; cu_seqlens: device int32[batch+1]; out: device, dense
 * [batch][heads][t_pad][depth].  Sequences longer than t_pad are clipped.
 */
SBT_API sbt_status sbt_ragged_tile_load(sbt_context* ctx, sbt_dtype dtype, const void* x, int64_t total_rows, int32_t heads,
                                int32_t depth, int64_t ld_row, int64_t ld_head, const int32_t* cu_seqlens,
                                int32_t batch, int32_t t_pad, void* out, void* stream);

/*
 * Ragged 3D tile store: the inverse of sbt_ragged_tile_load.
 * Mojo "RaggedTMA3DTile", async_copy_from_col / async_copy_batched: tiles go
 * back to the packed ragged array, only the first `dynamic_dim` rows of a tile
 * (valid sequence positions) are written, and what overhangs is masked off.
 *
 *   x[(cu[b]+r)*ld_row + h*ld_head + d] = tiles[((b*heads + h)*t_pad + r)*depth + d]
 *     for r < min(cu[b+1]-cu[b], t_pad) with 0 <= cu[b]+r < total_rows;
 *   every other element of x keeps its bits.
 *
 * tiles: device, dense [batch][heads][t_pad][depth]; cu_seqlens: device
 * int32[batch+1]; x: device packed [total_rows] rows with strides (ld_row,
 * ld_head), both positive.  Sequences whose packed rows overlap get one of the
 * candidate values (undefined which).
 */
SBT_API sbt_status sbt_ragged_tile_store(sbt_context* ctx, sbt_dtype dtype, const void* tiles, int32_t batch,
                                         int32_t heads, int32_t depth, int32_t t_pad, const int32_t* cu_seqlens,
                                         void* x, int64_t total_rows, int64_t ld_row, int64_t ld_head, void* stream);

/*
 * Boundary-tile GEMM  C = A * B.
 * cuTile.jl "Operations", muladd: (M,K) x (K,N) -> (M,N) with bf16 inputs
 * accumulating in fp32.  Tylo.jl "Boundary tiles", section "Accumulator
 * stores and GEMM": ceiling-division K loop and output grid, boundary tiles
 * zero-filled, the fp32 accumulator converted to the output type at the store
 * (round to nearest even) and stores outside M x N suppressed.
 *
 * A: device bf16, M x K, row stride lda >= K.  B: device bf16, K x N, row
 * stride ldb >= N.  C: device, M x N, row stride ldc >= N, c_dtype SBT_BF16
 * or SBT_F32.  Any leading dimension is accepted (odd ones included); C
 * elements outside M x N (padding columns) are never written.
 * workspace: device scratch of at least sbt_gemm_bounded_workspace_size()
 * bytes, 256-byte aligned, owned by the caller; it holds re-laid-out copies of
 * A and B and may be reused once the call has completed on `stream`.
 */
SBT_API sbt_status sbt_gemm_bounded_workspace_size(sbt_context* ctx, int64_t M, int64_t N, int64_t K, int64_t lda,
                                           int64_t ldb, size_t* bytes);
SBT_API sbt_status sbt_gemm_bounded(sbt_context* ctx, const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
                            int64_t ldc, sbt_dtype c_dtype, int64_t M, int64_t N, int64_t K, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * Block-scaled GEMM  D = (A .* a_scale) * (B .* b_scale) + acc.
 * cuTile.jl "Operations", muladd_scaled: A (M x K) and B (K x N) in a
 * low-precision float format, a_scale (M x K_s) and b_scale (K_s x N) in
 * E8M0 or E4M3; scale element j of a row of a_scale (of a column of b_scale)
 * multiplies the contiguous block of K / K_s elements k = j*K/K_s ..
 * (j+1)*K/K_s - 1 of that row of A (column of B).  fp32 accumulator, fp32
 * acc and D.
 *
 * Formats (OCP 8-bit floating point and microscaling formats):
 *   SBT_FMT_E4M3  1-4-3, bias 7, no infinities, S.1111.111 is NaN
 *   SBT_FMT_E5M2  1-5-2, bias 15, IEEE infinities and NaNs
 *   SBT_FMT_E8M0  unsigned power of two 2^(e-127), 0xFF is NaN (scales only)
 *   SBT_FMT_E2M1  4-bit 1-2-1, bias 1, values 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *                 (operands only); two per byte, element i of a row-major
 *                 array (i = row * ld + col) in byte i / 2, the even element
 *                 in the low nibble; ld must be even.
 *
 * a_fmt, b_fmt: E4M3, E5M2 or E2M1 (they may differ).  s_fmt: E8M0 or E4M3,
 * both scale arrays.  A: device, row stride lda >= K (elements).  B: device,
 * row stride ldb >= N.  a_scale: device bytes, row stride ld_sa >= K_s.
 * b_scale: device bytes, row stride ld_sb >= N.  K_s >= 1 must divide K
 * (K_s is ignored when K = 0).  acc: device fp32, row stride ld_acc >= N, or
 * NULL for zero; it may be D itself (then ld_acc == ldd) but may not
 * otherwise overlap D.  D: device fp32, row stride ldd >= N; elements outside
 * M x N are never written.
 *
 * Accuracy: each scaled operand value (code value times its scale) is formed
 * exactly and the products are summed in fp32, provided every scaled operand
 * lies in the normal range of bf16/fp32 (E8M0 scale exponents from 2^-124 to
 * 2^119 with E4M3 operands; any E4M3 scale).  NaN codes propagate to the row
 * (A, a_scale) or column (B, b_scale) of D they feed.
 *
 * Paths: under SBT_PATH_AUTO or SBT_PATH_TMA the call runs on the tensor
 * cores' block scaling when the formats allow it: E2M1 x E2M1 with E8M0 scales
 * and K / K_s = 32 on tcgen05.mma kind::mxf4 (packed 4-bit operands), E2M1 x
 * E2M1 with E4M3 scales and K / K_s = 16 on kind::mxf4nvf4 (the scales' signs
 * are moved onto the operand codes first), and any other mix of E4M3 / E5M2 /
 * E2M1 with E8M0 scales and K / K_s = 32 on kind::mxf8f6f4 (8-bit staging).
 * Every other combination, and any combination under SBT_PATH_SCALAR or
 * SBT_PATH_VECTOR, stages the scaled operands as bf16 for the bf16
 * tensor-core kernel.  The paths meet the same accuracy statement; they may
 * differ in the order of the fp32 sums.
 *
 * workspace: device scratch of at least sbt_gemm_block_scaled_workspace_size()
 * bytes (enough for either path), 256-byte aligned, owned by the caller
 * (re-laid-out copies of the operands and scales).
 */
typedef enum { SBT_FMT_E4M3 = 0, SBT_FMT_E5M2 = 1, SBT_FMT_E8M0 = 2, SBT_FMT_E2M1 = 3 } sbt_lowp_format;
SBT_API sbt_status sbt_gemm_block_scaled_workspace_size(sbt_context* ctx, int64_t M, int64_t N, int64_t K,
                                                        size_t* bytes);
SBT_API sbt_status sbt_gemm_block_scaled(sbt_context* ctx, sbt_lowp_format a_fmt, const void* A, int64_t lda,
                                         sbt_lowp_format b_fmt, const void* B, int64_t ldb, sbt_lowp_format s_fmt,
                                         const void* a_scale, int64_t ld_sa, const void* b_scale, int64_t ld_sb,
                                         int64_t K_s, const float* acc, int64_t ld_acc, float* D, int64_t ldd,
                                         int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                                         void* stream);

/*
 * Boundary-tile GEMM without any device allocation.
 * The pages have no counterpart to this call; it exists for callers that
 * cannot allocate device memory when they multiply: plugins confined to
 * another framework's memory pool (they may not call the CUDA allocator
 * themselves), code running under a device-memory budget committed up front,
 * and latency-critical paths that cannot take the implicit device
 * synchronisation of cudaMalloc and cudaFree.
 *
 * Same arguments and result as sbt_gemm_bounded, minus the workspace: the
 * operand-staging scratch is a fixed array of SBT_GEMM_NOALLOC_SCRATCH_BYTES
 * inside the library (one per device, held from module load until process
 * exit).  Shapes whose sbt_gemm_bounded_workspace_size() exceeds that size
 * are rejected with SBT_ERR_INVALID_ARG before anything is launched.  The
 * call itself allocates nothing (no cudaMalloc, no cudaFree, no allocating
 * library routine).
 *
 * Set-up: the first call on a device (whatever its shape) looks up the
 * array's device address with cudaGetSymbolAddress, with that device current,
 * and caches it; make that first call before any stream capture.  Like every
 * call of this library it leaves ctx's device current on the calling thread.
 * All calls share the one array and it keeps the previous call's contents
 * (the call rewrites every byte it reads, so nothing needs clearing); calls
 * that can overlap on the GPU -- different streams, or unsynchronised host
 * threads -- race on it.
 */
#define SBT_GEMM_NOALLOC_SCRATCH_BYTES (16u << 20)
SBT_API sbt_status sbt_gemm_bounded_noalloc(sbt_context* ctx, const void* A, int64_t lda, const void* B, int64_t ldb,
                                            void* C, int64_t ldc, sbt_dtype c_dtype, int64_t M, int64_t N, int64_t K,
                                            void* stream);

/*
 * A paged key-value cache, the attention that reads it, and the pass that
 * fills it.
 *
 * The cache holds, for every sequence, the keys and values of its positions
 * 0 .. len - 1 in fixed-size pages drawn from a common pool.  Position t of
 * sequence s lies in slot t % page_size of page page_table[s*ld_table +
 * t / page_size].  A page number outside [0, n_pages) (such as the -1 of a row
 * not yet filled) is no page: its positions are masked on a read and dropped
 * on a write, as out-of-range indices are by the gather and the scatter.
 */

/* Pages of the sequences, and who holds them.  All arrays are device memory. */
typedef struct {
    int32_t* page_table;  /* [n_seq][ld_table], the first max_pages columns are used */
    int64_t ld_table;     /* >= max_pages */
    int32_t n_seq, max_pages;
    int32_t* lens;        /* [n_seq] positions held; taken as min(max(len, 0), max_pages * page_size) */
    int64_t n_pages;      /* pages of the pool, < 2^31 */
    int32_t page_size;    /* positions per page, >= 1 */
    int32_t* refs;        /* [n_pages] holders of each page, 0: free; may be NULL where a call does not need it */
} sbt_page_map;

/* Keys and values of one layer.  Element (page, slot, head, d) of either lies
 * at page*ld_page + slot*ld_slot + head*ld_head + d: any order of slots and
 * heads within a page, and pages spaced at will. */
typedef struct {
    void *k, *v;               /* device, `dtype` of the call */
    int32_t heads, head_dim;   /* key-value heads; elements of a head */
    int64_t ld_page, ld_slot, ld_head;
} sbt_kv_cache;

/*
 * Attention of one new token per sequence over the cache.
 *
 *   visible(b) = positions t of sequence s = seq[b] (s = b if seq is NULL) with
 *                max(0, len - window) <= t < len (0 <= t < len if window is 0)
 *                on a page of the pool (and t < 2^31 - 1024)
 *   score[t]   = scale * sum_d q[b][h][d] * K[t][h / (q_heads / heads)][d]
 *   out[b][h]  = sum_t softmax(score)[t] * V[t][h / (q_heads / heads)]
 *   lse[b][h]  = log(sum_t exp(score[t]))
 *
 * for b < batch, h < q_heads.  A row that sees no position (length 0, seq[b]
 * outside [0, n_seq), no mapped page), or whose scores are all minus infinity,
 * gets out = 0 and lse = minus infinity.  Cache contents at positions that are
 * not visible are never read: NaN there reaches nothing.  A score of plus
 * infinity or NaN gives NaN in its row; an infinite V at a visible position
 * gives infinity or NaN in its column.  out must not overlap q or the cache.
 *
 * dtype: of q, the cache and out.  Products and sums are fp32; with SBT_BF16
 * and SBT_F16 a probability enters the second product as the sum of two 16-bit
 * numbers, 16 and 22 significant bits (with SBT_F16 in steps of 2^-39 of the
 * row's largest one at least).  1 <= head_dim <= 256; cache->heads divides q_heads.
 * q, out: strides in elements per batch entry (ld_q, ld_out) and head (ld_qh,
 * ld_oh).  lse: device fp32, dense [batch][q_heads], or NULL.
 * workspace: device scratch of sbt_paged_attention_workspace_size() bytes,
 * 256-byte aligned, owned by the caller and free again once the call has
 * completed on `stream`; its size depends on neither the batch nor the
 * lengths.  refs may be NULL.
 */
SBT_API sbt_status sbt_paged_attention_workspace_size(sbt_context* ctx, int32_t q_heads, int32_t kv_heads,
                                                      int32_t head_dim, size_t* bytes);
SBT_API sbt_status sbt_paged_attention(sbt_context* ctx, sbt_dtype dtype, const void* q, int64_t ld_q, int64_t ld_qh,
                                       int32_t batch, int32_t q_heads, const sbt_kv_cache* cache,
                                       const sbt_page_map* map, const int32_t* seq, float scale, int32_t window,
                                       void* out, int64_t ld_out, int64_t ld_oh, float* lse, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* Pairs that a rotation turns: (i, i + rot_dim/2), or (2i, 2i + 1). */
typedef enum { SBT_ROPE_HALF = 0, SBT_ROPE_INTERLEAVED = 1 } sbt_rope_layout;
/* How the frequencies f_i = base^(-2i/rot_dim) are stretched by `factor` s for
 * contexts longer than the model was trained on:
 *   SBT_ROPE_NONE      f_i
 *   SBT_ROPE_LINEAR    f_i / s
 *   SBT_ROPE_NTK       (base * s^(rot_dim/(rot_dim-2)))^(-2i/rot_dim)
 *   SBT_ROPE_BY_PARTS  (1-g) f_i / s + g f_i with g = clamp((n_i - low)/(high - low), 0, 1)
 *                      and n_i = orig_len * f_i / (2 pi), the turns made within the trained length */
typedef enum { SBT_ROPE_NONE = 0, SBT_ROPE_LINEAR = 1, SBT_ROPE_NTK = 2, SBT_ROPE_BY_PARTS = 3 } sbt_rope_scaling;

/* Rotations of the positions [0, n_pos): pair i at position t by the angle
 * whose cosine and sine are table[(t*rot_dim/2 + i)*2 + {0, 1}] (device fp32,
 * 8-byte aligned).  rot_dim = 0 (or a NULL sbt_rope): nothing is turned and
 * any position >= 0 is legal. */
typedef struct {
    const float* table;
    int64_t n_pos;
    int32_t rot_dim;   /* even, <= head_dim: the first rot_dim elements of a head are turned */
    int32_t layout;    /* sbt_rope_layout */
} sbt_rope;

/* Fills table[n_pos][rot_dim/2][2] (2^40 pairs at most) with amplitude * (cos,
 * sin)(t * f_i), angles formed in 64 bits and rounded once.  base > 0, factor > 0; low, high and
 * orig_len are read by SBT_ROPE_BY_PARTS only (high > low, orig_len > 0). */
SBT_API sbt_status sbt_rope_table(sbt_context* ctx, float* table, int64_t n_pos, int32_t rot_dim, double base,
                                  sbt_rope_scaling scaling, double factor, int64_t orig_len, double low, double high,
                                  double amplitude, void* stream);

/*
 * Per-head norm of queries and keys with the position rotation in the same
 * pass, and the append of keys and values to the cache.
 *
 * For each head row x (head_dim elements) of q with weight w = q_weight, and
 * of k with w = k_weight:
 *   n = x * w / sqrt(mean(x^2) + eps)     (n = x where the weight is NULL)
 *   y = n with its first rot_dim elements turned by the table at positions[t]
 * computed in fp32 and rounded once.  y of q goes to q_out, y of k to k_out
 * (may be NULL with a cache) and, with a cache, to position positions[t] of
 * sequence seq[t] (t if seq is NULL); the rows of v (NULL: none) go there as
 * they are.  A token whose position is negative or, where something is turned,
 * at or past n_pos is padding: its rows of q_out and k_out are zero and the
 * cache is not written.  A position without a page (or past max_pages *
 * page_size, or a sequence outside [0, n_seq)) is not written to the cache.
 * Two tokens of one call at the same place get one of the candidate values.
 * map->lens and map->refs are neither read nor written (may be NULL).
 *
 * q, k, v: device [tokens] rows with element strides (ld_*, ld_*h) per token
 * and head, so that they may be parts of one packed projection; k and v have
 * k_heads heads.  q_out may be q and k_out may be k (same strides).
 * 1 <= head_dim <= 512; with a cache, cache->heads = k_heads and
 * cache->head_dim = head_dim.  k_heads = 0 or q_heads = 0 leaves that part out;
 * q_heads + 2 k_heads is at most 2^30.
 */
SBT_API sbt_status sbt_qk_norm_rope(sbt_context* ctx, sbt_dtype dtype, const void* q, int64_t ld_q, int64_t ld_qh,
                                    const void* k, int64_t ld_k, int64_t ld_kh, int64_t tokens, int32_t q_heads,
                                    int32_t k_heads, int32_t head_dim, const int32_t* positions, const sbt_rope* rope,
                                    const void* q_weight, const void* k_weight, float eps, void* q_out,
                                    int64_t ld_qo, int64_t ld_qoh, void* k_out, int64_t ld_ko, int64_t ld_koh,
                                    const void* v, int64_t ld_v, int64_t ld_vh, const sbt_kv_cache* cache,
                                    const sbt_page_map* map, const int32_t* seq, void* stream);

/*
 * Gradient of sbt_qk_norm_rope.  gq, gk: gradients of q_out and k_out; q, k:
 * the forward call's inputs (not read, and may be NULL, where the weight is
 * NULL).  dq, dk get the gradients of q and k in `dtype` (rows of padding
 * tokens are zero; dq may be gq and dk may be gk); dq_weight, dk_weight (fp32
 * [head_dim], required exactly where the weight is given) the weights', summed
 * over tokens and heads in fp32 in an order that is fixed on one device.
 * workspace as elsewhere, of sbt_qk_norm_rope_backward_workspace_size() bytes.
 */
SBT_API sbt_status sbt_qk_norm_rope_backward_workspace_size(sbt_context* ctx, int32_t head_dim, size_t* bytes);
SBT_API sbt_status sbt_qk_norm_rope_backward(sbt_context* ctx, sbt_dtype dtype, const void* gq, int64_t ld_gq,
                                             int64_t ld_gqh, const void* gk, int64_t ld_gk, int64_t ld_gkh,
                                             const void* q, int64_t ld_q, int64_t ld_qh, const void* k, int64_t ld_k,
                                             int64_t ld_kh, int64_t tokens, int32_t q_heads, int32_t k_heads,
                                             int32_t head_dim, const int32_t* positions, const sbt_rope* rope,
                                             const void* q_weight, const void* k_weight, float eps, void* dq,
                                             int64_t ld_dq, int64_t ld_dqh, void* dk, int64_t ld_dk, int64_t ld_dkh,
                                             float* dq_weight, float* dk_weight, void* workspace,
                                             size_t workspace_bytes, void* stream);

/*
 * Pages of a cache: copy, reserve, fork, free, compact.
 *
 * A pool is where pages of one kind lie: page p of plane i (a layer, say) is
 * the page_bytes bytes at base + i*plane_stride + p*page_stride.  A page number
 * stands for that page in every plane of every pool of the call, so one page
 * map can serve all layers' keys and values.  Strides and sizes are in bytes;
 * pages of 16-byte-aligned addresses and sizes move as 16-byte vectors.
 *
 * All state is on the device, and what a call does follows from it alone: free
 * pages (refs 0 or less) are given lowest number first, and requests are
 * served in their order.  Requests that are not legal (numbers out of range,
 * no page left) are left out; nothing faults.
 */
#define SBT_MAX_PAGE_POOLS 64
typedef struct {
    void* base;
    int64_t n_planes, plane_stride, page_stride, page_bytes;
} sbt_page_pool;

/* Scratch of reserve, fork and compact (256-byte aligned, the caller's). */
SBT_API sbt_status sbt_pages_workspace_size(sbt_context* ctx, int32_t n_seq, int64_t n_pages, size_t* bytes);

/* Copies page src[i] to page dst[i], i < n.  Pairs with a number outside
 * [0, n_pages) are left out.  A page that is both a source and a destination,
 * or twice a destination, holds one of the candidates per 16 bytes. */
SBT_API sbt_status sbt_pages_copy(sbt_context* ctx, const sbt_page_pool* pools, int32_t n_pools, int64_t n_pages,
                                  const int32_t* src, const int32_t* dst, int64_t n, void* stream);

/* Grows every sequence s with target[s] > lens[s] to target[s] positions (lens
 * is set): the table's next entries get free pages with one holder each.
 * Where the last page held is part full and has other holders, the sequence
 * first gets a copy of its own (of pools' bytes), so that what it appends
 * reaches no other sequence.  Pages go to sequences in their order; one whose
 * pages do not all fit after those of the sequences before it, or that has no
 * room in its row, keeps its length (as lens then shows). */
SBT_API sbt_status sbt_pages_reserve(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools,
                                     int32_t n_pools, const int32_t* target, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Forks sequence from[i] into sequence to[i], i < n <= n_seq: the child shares
 * the full pages and gets a copy of a part-full last page.  Left out (the
 * child stays as it is): numbers out of range, from[i] = to[i], an empty
 * parent, a child that is not empty or that an earlier pair took, and pairs
 * that no free page is left for. */
SBT_API sbt_status sbt_pages_fork(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools,
                                  int32_t n_pools, const int32_t* from, const int32_t* to, int32_t n,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Cuts sequence seqs[i] to at most keep[i] positions (0 if keep is NULL): the
 * pages past them lose a holder, their table entries become -1, lens is set. */
SBT_API sbt_status sbt_pages_free(sbt_context* ctx, const sbt_page_map* map, const int32_t* seqs, const int32_t* keep,
                                  int32_t n, void* stream);

/* Packs the held pages (refs > 0) into the lowest numbers: with L of them, the
 * k-th held page at L or above moves to the k-th hole below L.  page_to[p]
 * (int32 [n_pages]) gets p's new number or -1, n_live (int32 [1]) gets L,
 * refs_out ([n_pages]) the holders by new number and table_out ([n_seq]
 * [ld_out]) the entries within each length by new number (entries past it are
 * not written).  table_out may be the map's table (then ld_out = ld_table) and
 * refs_out the map's refs; otherwise the map is left as it was.  Bytes of pages
 * that move stay at their old place too. */
SBT_API sbt_status sbt_pages_compact(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools,
                                     int32_t n_pools, int32_t* table_out, int64_t ld_out, int32_t* refs_out,
                                     int32_t* page_to, int32_t* n_live, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * Slot maps: what a step's calls read about its new tokens, from the requests'
 * lengths.  Entry b of the batch (sequence s = seqs[b], or b where seqs is NULL)
 * brings n = max(n_new[b], 0) tokens; the tokens of all entries follow one
 * another.  The tokens of entry b stand at positions first .. first + n - 1 of
 * its sequence, with first = start[b] or, where start is NULL, lens[s] - n (they
 * are the last of what the sequence holds, as after sbt_pages_reserve).
 *
 *   cu[b]         tokens before entry b, cu[batch] all; at most capacity
 *   seq[t]        the token's sequence
 *   positions[t]  its position
 *   slots[t]      page * page_size + slot of its position in the pool
 *   last[b]       the entry's last token
 *
 * for t < capacity, b < batch; outputs that are NULL are left out.  -1 stands in
 * seq, positions and slots of the places past the last token (padding, as every
 * call here reads it) and of tokens whose sequence is outside [0, n_seq); in
 * positions and slots where the position is negative or at 2^31 or more; in
 * slots where the position has no page; in last where the entry has no token or
 * its last one is past the capacity.  An entry that the capacity cuts has places
 * for its first tokens, at their positions, and none for the others, which its
 * sequence then lacks; sbt_paged_tree_attention would take those places for the
 * sequence's last tokens, so choose a capacity for all tokens, or give the attention
 * a seq outside [0, n_seq) for that entry.  slots needs n_pages * page_size <= 2^31.
 * map->refs is not needed, map->lens only where start is NULL.
 */
SBT_API sbt_status sbt_pages_slots(sbt_context* ctx, const sbt_page_map* map, const int32_t* n_new, int32_t batch,
                                   const int32_t* seqs, const int32_t* start, int32_t capacity, int32_t* cu,
                                   int32_t* seq, int32_t* positions, int32_t* slots, int32_t* last, void* stream);

/*
 * Trees of drafted tokens: entry b's tokens are the rows cu[b] .. cu[b+1] - 1
 * (cu ascending), parents[row] is the number within the entry of the token that
 * the row's token continues, an earlier one; any other value (such as -1) makes
 * it continue the sequence itself.
 *
 *   mask[row * ld_mask + w], bit j: token 32 w + j of the entry is the row's token
 *                 or one of its ancestors (w < ld_mask; later tokens have no bit)
 *   turned[row]   positions[row] less what siblings count twice: the position of
 *                 the entry's first token plus the token's depth in its tree, by
 *                 which its query and key are turned; -1 where positions[row] < 0
 *
 * for row < rows.  mask or turned may be NULL; positions is read for turned only.
 * Rows of no entry get no bits and -1.
 */
SBT_API sbt_status sbt_tree_plan(sbt_context* ctx, const int32_t* parents, const int32_t* cu, int32_t batch,
                                 int32_t rows, const int32_t* positions, int32_t* turned, int32_t* mask,
                                 int64_t ld_mask, void* stream);

/*
 * Attention of several new tokens per sequence over the cache, which holds them
 * already: a prompt's next piece, or a tree of drafted tokens.
 *
 * Entry b's tokens are the rows cu[b] .. cu[b+1] - 1 of q and out, n of them; with
 * L the length of sequence s = seq[b] (b where seq is NULL), token j of the entry
 * stands at position L - n + j: all n of them have to be there, so an entry that
 * sbt_pages_slots has cut at its capacity is not one to attend.  Token i sees the
 * positions t of its sequence on a page of the pool with
 *   0 <= t < L - n                 (what was held before), or
 *   t = L - n + j, t >= 0, j < n   and bit j of its mask row set (j <= i where mask is NULL).
 * Scores, out and lse are those of sbt_paged_attention over these positions;
 * lse is dense fp32 [rows][q_heads] or NULL.  Products and sums are fp32; a
 * probability enters the second product as the sum of two 16-bit numbers, 16
 * (SBT_BF16) and 22 (SBT_F16) significant bits, with SBT_F16 in steps of 2^-33 of
 * the row's largest one at least.  A token that
 * sees nothing gets zeros and minus infinity.  Contents at positions that a token
 * does not see reach none of its results, whatever they are; but all slots of the
 * pages that hold the entry's positions may be read, those past the length too,
 * so nothing may write them at the same time.  An entry with more than max_new
 * tokens, or with rows outside [0, rows), is left out; rows of no entry and of
 * entries left out are not written.
 *
 * dtype: SBT_BF16 or SBT_F16.  mask: int32 [rows][ld_mask], bit 32 w + j as
 * sbt_tree_plan writes it (tokens from 32 ld_mask on are seen by none).
 * 1 <= head_dim <= 256, cache->heads divides q_heads, max_new * (q_heads /
 * cache->heads) < 2^24.  workspace as for sbt_paged_attention; its size depends
 * on neither the batch nor the lengths, and serves every smaller max_new.
 */
SBT_API sbt_status sbt_paged_tree_attention_workspace_size(sbt_context* ctx, int32_t max_new, int32_t q_heads,
                                                           int32_t kv_heads, int32_t head_dim, size_t* bytes);
SBT_API sbt_status sbt_paged_tree_attention(sbt_context* ctx, sbt_dtype dtype, const void* q, int64_t ld_q,
                                            int64_t ld_qh, int32_t rows, const int32_t* cu, int32_t batch,
                                            int32_t max_new, int32_t q_heads, const sbt_kv_cache* cache,
                                            const sbt_page_map* map, const int32_t* seq, float scale,
                                            const int32_t* mask, int64_t ld_mask, void* out, int64_t ld_out,
                                            int64_t ld_oh, float* lse, void* workspace, size_t workspace_bytes,
                                            void* stream);

/*
 * Root-mean-square norm of rows with the residual's addition:
 *
 *   h = x + r (x where r is NULL),   y = h * weight / sqrt(mean(h^2) + eps)
 *
 * per row of `cols` elements, in fp32 (weight NULL: 1); h_out and y get h and y,
 * each rounded once, and codes (where given) y in 8 bits with a scale per block
 * of columns, which is what sbt_gemm_block_scaled reads as A and a_scale with
 * K_s = cols / block (a mean of squares past fp32's range makes y zero; one of zero
 * with eps = 0 divides by zero):
 *
 *   scales[row][j] = 2^e, the least power of two (2^-124 at least; 1 for a block of
 *                    zeros) with which no |y| of columns j*block .. (j+1)*block - 1
 *                    passes largest * 2^e, largest = 448 (E4M3) or 57344 (E5M2), as E8M0
 *   codes[row][c]  = y / 2^e to nearest even; a block that holds an infinity or NaN
 *                    gets the scale NaN (0xFF) and NaN codes
 *
 * h_out, y and codes may be NULL, but not both y and codes.  h_out or y (not
 * both) may be x or r itself (same stride).  Strides in elements, at least cols
 * for what is written; 1 <= cols <= 2^24, rows < 2^31.
 */
typedef struct {
    void* codes;         /* [rows][ld] bytes, ld >= cols */
    int64_t ld;
    uint8_t* scales;     /* [rows][ld_scale] bytes, ld_scale >= cols / block */
    int64_t ld_scale;
    int32_t format;      /* SBT_FMT_E4M3 or SBT_FMT_E5M2 */
    int32_t block;       /* 16, 32, 64 or 128; divides cols */
} sbt_code_rows;
SBT_API sbt_status sbt_add_rms_norm(sbt_context* ctx, sbt_dtype dtype, const void* x, int64_t ld_x, const void* r,
                                    int64_t ld_r, int64_t rows, int32_t cols, const void* weight, float eps,
                                    void* h_out, int64_t ld_h, void* y, int64_t ld_y, const sbt_code_rows* codes,
                                    void* stream);

/*
 * Gradient of sbt_add_rms_norm at h (its h_out, or x where there is no r): with
 * gy the gradient of y and gh that of h_out (NULL: zero), dx gets the gradient
 * of h, which is that of x and of r (a row that was added to all, with a stride of
 * zero, has the sum of dx over the rows), in `dtype`, and dweight (fp32 [cols],
 * required exactly where weight is given) the weight's, summed over the rows in
 * fp32 in an order that is fixed on one device.  dx may be gy, gh or h (same
 * stride).  workspace as elsewhere, of
 * sbt_add_rms_norm_backward_workspace_size() bytes.
 */
SBT_API sbt_status sbt_add_rms_norm_backward_workspace_size(sbt_context* ctx, int64_t rows, int32_t cols,
                                                            size_t* bytes);
SBT_API sbt_status sbt_add_rms_norm_backward(sbt_context* ctx, sbt_dtype dtype, const void* gy, int64_t ld_gy,
                                             const void* gh, int64_t ld_gh, const void* h, int64_t ld_h, int64_t rows,
                                             int32_t cols, const void* weight, float eps, void* dx, int64_t ld_dx,
                                             float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * A few rows times a matrix of 4-bit weights with group scales, the B operand of
 * sbt_gemm_block_scaled as it stands there (E2M1 codes, K x N, two columns a byte,
 * ldb even; scales K_s x N in E8M0 or E4M3, one per K / K_s weights of a column):
 *
 *   y[t][n] = alpha * sum_k x[t][k] * B[k][n] * b_scale[k / (K / K_s)][n]
 *
 * for t < tokens, n < N.  dtype: of x; y_dtype: of y, SBT_F32, SBT_BF16 or
 * SBT_F16.  K_s divides K and K / K_s is a multiple of 16; tokens <= 65535 * 8
 * (the weights are read once per 16 of them).  Sums are fp32, in an order that is
 * fixed on one device; a row of x enters the products exactly with SBT_F16, and
 * with SBT_BF16 and SBT_F32 as one and two fp16 numbers scaled by a power of two:
 * off by at most 2^-39 of its largest finite |x| (and, SBT_F32, 2^-21 of itself).
 * The sums are those of the scaled numbers, the largest below 2^15: group scales from
 * 2^108 on may take them past fp32's range although the result would not be.  An
 * infinity or NaN in x reaches its own row only; a NaN scale (E8M0 0xFF, E4M3
 * 0x7F and 0xFF) its own column.
 */
SBT_API sbt_status sbt_matvec_e2m1(sbt_context* ctx, sbt_dtype dtype, const void* x, int64_t ld_x, int64_t tokens,
                                   const void* B, int64_t ldb, sbt_lowp_format s_fmt, const void* b_scale,
                                   int64_t ld_sb, int64_t K_s, float alpha, void* y, int64_t ld_y, sbt_dtype y_dtype,
                                   int64_t N, int64_t K, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SBT_H_ */
