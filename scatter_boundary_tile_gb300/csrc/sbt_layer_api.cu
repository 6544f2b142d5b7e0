// C ABI of a decoding layer's operators around the attention: argument
// validation and dispatch.  Every check here runs before any launch; a failing
// call launches nothing.
#include "sbt_checks.cuh"

namespace {

using namespace sbt_checks;

// Rows of a matrix that is read (or, with `write`, written).
sbt_status check_rows(const SbtRows& m, int64_t rows, int64_t cols, int es, bool write, const char* name,
                      const char* what) {
    auto row = [&](const char* text) { return say(what, ": ") + name + text; };
    SBT_REQUIRE(m.p, row(" is NULL"));
    SBT_REQUIRE(m.ld >= 0, row(" has a negative stride"));
    SBT_REQUIRE(!write || rows <= 1 || m.ld >= cols, row(" stride smaller than its row"));
    SBT_REQUIRE_ALIGNED(m.p, es, row(" is not aligned to its element size"));
    return SBT_OK;
}

sbt_status check_extent(int64_t rows, int32_t cols, float eps, const char* what) {
    SBT_REQUIRE(rows >= 0 && rows < (1ll << 31), say(what, ": rows must be in [0, 2^31)"));
    SBT_REQUIRE(cols >= 1 && cols <= 1 << 24, say(what, ": cols must be in [1, 2^24]"));
    SBT_REQUIRE(eps >= 0.f, say(what, ": negative eps"));
    return SBT_OK;
}

}  // namespace

extern "C" {

sbt_status sbt_add_rms_norm(sbt_context* ctx, sbt_dtype dtype, const void* x, int64_t ld_x, const void* r,
                            int64_t ld_r, int64_t rows, int32_t cols, const void* weight, float eps, void* h_out,
                            int64_t ld_h, void* y, int64_t ld_y, const sbt_code_rows* codes, void* stream) {
    const char* const w = "add_rms_norm";
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_dtype(dtype, w));
    const int es = sbt_dtype_size(dtype);
    SBT_TRY(check_extent(rows, cols, eps, w));
    SBT_REQUIRE(y || codes, "add_rms_norm: y and codes are both NULL");
    if (codes) {
        if (codes->format != SBT_FMT_E4M3 && codes->format != SBT_FMT_E5M2)
            return sbt_fail(SBT_ERR_UNSUPPORTED, "add_rms_norm: codes must be E4M3 or E5M2");
        const int32_t b = codes->block;
        SBT_REQUIRE((b == 16 || b == 32 || b == 64 || b == 128) && cols % b == 0,
                    "add_rms_norm: block must be 16, 32, 64 or 128 and divide cols");
    }
    if (rows == 0) return SBT_OK;
    const SbtRows mx = {x, ld_x}, mr = {r, ld_r}, mh = {h_out, ld_h}, my = {y, ld_y};
    SBT_TRY(check_rows(mx, rows, cols, es, false, "x", w));
    if (r) SBT_TRY(check_rows(mr, rows, cols, es, false, "r", w));
    if (h_out) SBT_TRY(check_rows(mh, rows, cols, es, true, "h_out", w));
    if (y) SBT_TRY(check_rows(my, rows, cols, es, true, "y", w));
    SBT_REQUIRE(!h_out || h_out != y, "add_rms_norm: h_out and y are the same array");
    auto in_place = [&](const SbtRows& m) { return !m.p || ((m.p != x || m.ld == ld_x) && (m.p != r || m.ld == ld_r)); };
    SBT_REQUIRE(rows == 1 || (in_place(mh) && in_place(my)), "add_rms_norm: in place needs the same stride");
    SBT_REQUIRE_ALIGNED(weight, es, "add_rms_norm: weight is not aligned to its element size");
    if (codes) {
        SBT_TRY(check_rows({codes->codes, codes->ld}, rows, cols, 1, true, "codes", w));
        SBT_TRY(check_rows({codes->scales, codes->ld_scale}, rows, cols / codes->block, 1, true, "scales", w));
    }
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_add_norm(ctx, dtype, mx, mr, rows, cols, weight, eps, mh, my, codes, (cudaStream_t)stream);
}

sbt_status sbt_add_rms_norm_backward_workspace_size(sbt_context* ctx, int64_t rows, int32_t cols, size_t* bytes) {
    SBT_REQUIRE(ctx && bytes, "add_rms_norm_backward_workspace_size: NULL argument");
    SBT_TRY(check_extent(rows, cols, 0.f, "add_rms_norm_backward_workspace_size"));
    *bytes = sbt_add_norm_bwd_bytes(ctx, rows, cols);
    return SBT_OK;
}

sbt_status sbt_add_rms_norm_backward(sbt_context* ctx, sbt_dtype dtype, const void* gy, int64_t ld_gy, const void* gh,
                                     int64_t ld_gh, const void* h, int64_t ld_h, int64_t rows, int32_t cols,
                                     const void* weight, float eps, void* dx, int64_t ld_dx, float* dweight,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    const char* const w = "add_rms_norm_backward";
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_dtype(dtype, w));
    const int es = sbt_dtype_size(dtype);
    SBT_TRY(check_extent(rows, cols, eps, w));
    SBT_REQUIRE(!weight == !dweight,
                "add_rms_norm_backward: the weight's gradient is required exactly where the weight is given");
    if (rows == 0 && !dweight) return SBT_OK;
    const SbtRows mgy = {gy, ld_gy}, mgh = {gh, ld_gh}, mh = {h, ld_h}, mdx = {dx, ld_dx};
    if (rows > 0) {
        SBT_TRY(check_rows(mgy, rows, cols, es, false, "gy", w));
        SBT_TRY(check_rows(mh, rows, cols, es, false, "h", w));
        if (gh) SBT_TRY(check_rows(mgh, rows, cols, es, false, "gh", w));
        SBT_TRY(check_rows(mdx, rows, cols, es, true, "dx", w));
        SBT_REQUIRE(rows == 1 || ((dx != gy || ld_dx == ld_gy) && (dx != gh || ld_dx == ld_gh) && (dx != h || ld_dx == ld_h)),
                    "add_rms_norm_backward: in place needs the same stride");
    }
    SBT_REQUIRE_ALIGNED(weight, es, "add_rms_norm_backward: weight is not aligned to its element size");
    SBT_REQUIRE_ALIGNED(dweight, 4, "add_rms_norm_backward: dweight is not 4-byte aligned");
    const size_t need = sbt_add_norm_bwd_bytes(ctx, rows, cols);
    if (need) SBT_TRY(check_workspace(workspace, workspace_bytes, need, w));
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_add_norm_bwd(ctx, dtype, mgy, mgh, mh, rows, cols, weight, eps, mdx, dweight, workspace,
                                   (cudaStream_t)stream);
}

sbt_status sbt_matvec_e2m1(sbt_context* ctx, sbt_dtype dtype, const void* x, int64_t ld_x, int64_t tokens,
                           const void* B, int64_t ldb, sbt_lowp_format s_fmt, const void* b_scale, int64_t ld_sb,
                           int64_t K_s, float alpha, void* y, int64_t ld_y, sbt_dtype y_dtype, int64_t N, int64_t K,
                           void* stream) {
    const char* const w = "matvec_e2m1";
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_dtype(dtype, w));
    SBT_TRY(check_dtype(y_dtype, w));
    if (s_fmt != SBT_FMT_E8M0 && s_fmt != SBT_FMT_E4M3)
        return sbt_fail(SBT_ERR_UNSUPPORTED, "matvec_e2m1: scales must be E8M0 or E4M3");
    SBT_REQUIRE(tokens >= 0 && N >= 0 && K >= 0, "matvec_e2m1: negative extent");
    SBT_REQUIRE(tokens <= 65535 * 8 && N < (1ll << 31) && K < (1ll << 31), "matvec_e2m1: extent too large");
    SBT_REQUIRE(ldb % 2 == 0 && ldb >= N, "matvec_e2m1: ldb must be even and at least N");
    if (tokens == 0 || N == 0) return SBT_OK;
    SBT_TRY(check_rows({y, ld_y}, tokens, N, sbt_dtype_size(y_dtype), true, "y", w));
    if (K > 0) {
        SBT_REQUIRE(K_s >= 1 && K % K_s == 0, "matvec_e2m1: K_s must divide K");
        if (K / K_s % 16) return sbt_fail(SBT_ERR_UNSUPPORTED, "matvec_e2m1: K / K_s must be a multiple of 16");
        SBT_TRY(check_rows({x, ld_x}, tokens, K, sbt_dtype_size(dtype), false, "x", w));
        SBT_REQUIRE(B, "matvec_e2m1: B is NULL");
        SBT_REQUIRE(b_scale, "matvec_e2m1: b_scale is NULL");
        SBT_REQUIRE(K_s == 1 || ld_sb >= N, "matvec_e2m1: ld_sb < N");
    }
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_matvec(ctx, dtype, {x, ld_x}, tokens, B, ldb, s_fmt == SBT_FMT_E4M3, b_scale, ld_sb, K_s, alpha,
                             {y, ld_y}, y_dtype, N, K, (cudaStream_t)stream);
}

}  // extern "C"
