// The entry points of products with 4-bit weights; their kernels are in layer_w4.h.
#include "layer_w4.h"
#include "layer_checks.h"

namespace dgt {

namespace {

thread_local struct {
  bool dense;
  W4Form form;
} g_w4_path;
void write_w4_path(std::string& to) {
  const W4Form& f = g_w4_path.form;
  to = std::string(g_w4_path.dense ? "linear_w4" : "grouped_w4") + " mfma w" + std::to_string(f.waves) + " t" +
       std::to_string(f.rows) + "x" + std::to_string(f.columns) + (f.whole ? "" : " through registers");
}

// Both entry points (G < 0: dense).
int run_w4(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, const int32_t* offsets, const void* A, int64_t lda,
           const void* B, int64_t ldb, int64_t stride_b, const void* scales, const void* zeros, int64_t lds,
           int64_t stride_s, int64_t group, const void* bias, int act, const void* R, int64_t ldr, void* Y, int64_t ldy,
           int out_dtype, void* stream) {
  const bool dense = G < 0;
  CHECK(check_dim("M", M));
  CHECK(check_dim("N", N));
  CHECK(check_dim("K", K));
  CHECK(check_dtype16(dtype));
  CHECK(check_out_dtype(dtype, out_dtype));
  CHECK(check_act(act));
  if (group < 32 || group % 32) return bad("%s=%lld is not a multiple of 32", "group", group);
  const int osz = out_dtype == GEMM_DTYPE_F32 ? 4 : 2;
  const int64_t g = dense ? 1 : G, runs = K / group + (K % group != 0);
  if (runs > kW4MaxRuns) return fail(GEMM_ERR_UNSUPPORTED, "more than 1536 groups of K values");
  if (ldb % 2) return bad("%s=%lld is odd: a row of codes starts in a byte's lower half", "ldb", ldb);
  if (!dense && g > 1) {
    if (stride_b < 0 || stride_b % 2) return bad("%s=%lld is negative or odd", "stride_b", stride_b);
    if (stride_s < 0) return bad("%s is negative: %lld", "stride_s", stride_s);
  }
  const Mat ma{"A", A, M, K, lda, 2}, mb{"B", B, N, (K + 1) / 2, ldb / 2, 1, g, stride_b / 2};
  const Mat ms{"scales", scales, N, runs, lds, 2, g, stride_s}, mz{"zeros", zeros, N, runs, lds, 2, g, stride_s};
  const Mat mbias{"bias", bias, 1, N, N, 2, g, N};
  const Mat mr{"R", R, M, N, ldr, osz}, my{"Y", Y, M, N, ldy, osz};
  const Mat moff{"offsets", offsets, 1, g + 1, g + 1, 4};
  CHECK(check_ld(ma));
  if (ldb < (K > 1 ? K : 1)) return bad("leading dimension of %s is %lld, smaller than %lld", "B", ldb, K > 1 ? K : 1);
  CHECK(check_ld(ms));
  CHECK(check_ld(my));
  if (R) CHECK(check_ld(mr));
  if (M == 0 || N == 0 || g == 0) {
    set_path("noop: empty output");
    return GEMM_OK;
  }
  CHECK(check_ptr(my));
  if (K > 0) {
    for (const Mat* m : {&ma, &mb, &ms}) CHECK(check_ptr(*m));
    if (zeros) CHECK(check_ptr(mz));
    for (const Mat* m : {&ma, &mb, &ms, &mz}) CHECK(check_apart(my, *m));
  }
  if (bias) CHECK(check_ptr(mbias));
  if (R) CHECK(check_ptr(mr));
  CHECK(check_apart(my, mbias));
  CHECK(check_apart_or_same(my, mr));
  if (!dense) {
    CHECK(check_ptr(moff));
    CHECK(check_apart(my, moff));
  }
  W4Args p{};
  LayerArgs& a = p.a;
  a.A = A;
  a.B = B;
  a.bias = bias;
  a.R = R;
  a.Y = Y;
  a.offsets = offsets;
  a.lda = lda;
  a.ldb = ldb / 2;
  a.ldr = ldr;
  a.ldy = ldy;
  a.stride_b = stride_b / 2;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.G = (int)g;
  a.mode = dense ? LAYER_DENSE : LAYER_ROWS;
  a.act = act;
  a.out32 = osz == 4;
  p.scales = scales;
  p.zeros = zeros;
  p.lds = lds;
  p.stride_s = stride_s;
  p.group = (int)(group < kMaxDim ? group : kMaxDim / 32 * 32);
  hipStream_t s = static_cast<hipStream_t>(stream);
  W4Form& form = g_w4_path.form;
  g_w4_path.dense = dense;
  const hipError_t e = dtype == GEMM_DTYPE_F16 ? launch_w4_f16(p, s, form) : launch_w4_bf16(p, s, form);
  if (form.many) return fail(GEMM_ERR_UNSUPPORTED, "too many output tiles for one launch");
  set_path_writer(write_w4_path);
  return launched(e);
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_linear_w4(int64_t M, int64_t N, int64_t K, int dtype, const void* A, int64_t lda, const void* B, int64_t ldb,
                   const void* scales, const void* zeros, int64_t lds, int64_t group, const void* bias, int act,
                   const void* R, int64_t ldr, void* Y, int64_t ldy, int out_dtype, void* stream) {
  return entry("linear_w4", M, N, K, [&] {
    return run_w4(-1, M, N, K, dtype, nullptr, A, lda, B, ldb, 0, scales, zeros, lds, 0, group, bias, act, R, ldr, Y,
                  ldy, out_dtype, stream);
  });
}

int gemm_grouped_w4(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, const int32_t* offsets, const void* A,
                    int64_t lda, const void* B, int64_t ldb, int64_t stride_b, const void* scales, const void* zeros,
                    int64_t lds, int64_t stride_s, int64_t group, const void* bias, int act, const void* R, int64_t ldr,
                    void* Y, int64_t ldy, int out_dtype, void* stream) {
  return entry("grouped_w4", M, N, K, [&] {
    CHECK(check_groups(G));
    return run_w4(G, M, N, K, dtype, offsets, A, lda, B, ldb, stride_b, scales, zeros, lds, stride_s, group, bias, act,
                  R, ldr, Y, ldy, out_dtype, stream);
  });
}

}  // extern "C"
