// Checks of arguments that the layer operators' entry points share, and what
// stands around each of their calls. A check returns GEMM_OK, or a code whose
// message it has recorded.
#pragma once

#include <cstdio>
#include <string>

#include "gemm_layer.h"
#include "api_state.h"
#include "layer_rows.h"

namespace dgt {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1024;
constexpr int64_t kMaxGroups = 65535;  // groups index a launch's second dimension

inline int bad(const char* fmt, const char* name, int64_t a, int64_t b = 0) {
  char buf[200];
  std::snprintf(buf, sizeof buf, fmt, name, (long long)a, (long long)b);
  return fail(GEMM_ERR_INVALID_ARG, buf);
}

// One matrix (or a stack of them) that a call reads or writes.
struct Mat {
  const char* name;
  const void* ptr;
  int64_t rows, cols, ld;
  int elem;                 // bytes
  int64_t count = 1, stride = 0;  // stacked matrices
  unsigned __int128 extent() const {
    if (!ptr || count <= 0) return 0;
    const unsigned __int128 one = extent_bytes(rows, cols, ld, elem);
    return one ? one + (unsigned __int128)(count - 1) * (unsigned __int128)stride * elem : 0;
  }
};

inline int check_dim(const char* name, int64_t v) {
  if (v < 0) return bad("negative dimension: %s=%lld", name, v);
  if (v > kMaxDim) return fail(GEMM_ERR_UNSUPPORTED, std::string(name) + " exceeds 2^31-1024");
  return GEMM_OK;
}
inline int check_ld(const Mat& m) {
  const int64_t least = m.cols > 1 ? m.cols : 1;
  if (m.ld < least) return bad("leading dimension of %s is %lld, smaller than %lld", m.name, m.ld, least);
  return GEMM_OK;
}
inline int check_ptr(const Mat& m) {
  if (!m.ptr) return fail(GEMM_ERR_INVALID_ARG, std::string(m.name) + " is NULL");
  if ((uintptr_t)m.ptr % m.elem)
    return bad("%s is not %lld-byte aligned", m.name, m.elem);
  return GEMM_OK;
}
inline int check_apart(const Mat& w, const Mat& r) {
  if (w.ptr && r.ptr && overlaps(w.ptr, w.extent(), r.ptr, r.extent()))
    return fail(GEMM_ERR_ALIAS, std::string(w.name) + " overlaps " + r.name);
  return GEMM_OK;
}
// As check_apart, but the two may be the same matrix.
inline int check_apart_or_same(const Mat& w, const Mat& r) {
  if (w.ptr == r.ptr && (w.ld == r.ld || w.rows <= 1) && w.elem == r.elem && w.stride == r.stride)
    return GEMM_OK;
  return check_apart(w, r);
}

#define CHECK(expr)                      \
  do {                                   \
    const int st_ = (expr);              \
    if (st_ != GEMM_OK) return st_;      \
  } while (0)

inline int check_dtype16(int dtype) {
  if (dtype == GEMM_DTYPE_F16 || dtype == GEMM_DTYPE_BF16) return GEMM_OK;
  char buf[96];
  std::snprintf(buf, sizeof buf, "dtype code %d is neither f16 (0) nor bf16 (1)", dtype);
  return fail(GEMM_ERR_UNSUPPORTED, buf);
}
inline int check_out_dtype(int dtype, int out) {
  if (out == dtype || out == GEMM_DTYPE_F32) return GEMM_OK;
  char buf[128];
  std::snprintf(buf, sizeof buf, "result dtype code %d is neither the operands' (%d) nor f32 (%d)",
                out, dtype, GEMM_DTYPE_F32);
  return fail(GEMM_ERR_UNSUPPORTED, buf);
}
inline int check_act(int act) {
  if (act >= GEMM_ACT_NONE && act <= GEMM_ACT_SILU) return GEMM_OK;
  return bad("%s code %lld is not one of GEMM_ACT_* (0 to 4)", "activation", act);
}

inline int check_groups(int64_t G) {
  if (G < 0) return bad("negative number of groups: %s=%lld", "G", G);
  if (G > kMaxGroups) return fail(GEMM_ERR_UNSUPPORTED, "G exceeds 65535");
  return GEMM_OK;
}

inline int launched(hipError_t e) {
  if (e == hipSuccess) return GEMM_OK;
  return fail(GEMM_ERR_HIP, std::string("kernel launch failed: ") + hipGetErrorString(e));
}

// Runs one entry point's work between the thread's state and the log, and
// keeps C++ exceptions (a failed allocation of a message) from crossing the C
// boundary.
template <class F>
inline int entry(const char* op, int64_t M, int64_t N, int64_t K, F work) noexcept {
  try {
    begin_call();
    const int st = work();
    log_layer_call(op, M, N, K, st);
    return st;
  } catch (...) {
    return GEMM_ERR_HIP;
  }
}

inline int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return GEMM_OK;
  if (have < need) return bad("%s of %lld bytes is smaller than the %lld needed", "workspace", have, need);
  if (!ws) return fail(GEMM_ERR_INVALID_ARG, "workspace is NULL");
  if ((uintptr_t)ws % 16) return fail(GEMM_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  return GEMM_OK;
}

inline int check_choices(int64_t T, int64_t top) {
  CHECK(check_dim("T", T));
  CHECK(check_dim("top", top));
  if (T * top > kMaxDim) return fail(GEMM_ERR_UNSUPPORTED, "T * top exceeds 2^31-1024");
  return GEMM_OK;
}
inline int check_rowtype(int dtype, int& rowtype, int& elem) {
  rowtype = dtype == GEMM_DTYPE_F32 ? ROW_F32 : dtype == GEMM_DTYPE_F16 ? ROW_F16 : ROW_BF16;
  elem = dtype == GEMM_DTYPE_F32 ? 4 : 2;
  if (dtype == GEMM_DTYPE_F32) return GEMM_OK;
  if (dtype == GEMM_DTYPE_F16 || dtype == GEMM_DTYPE_BF16) return GEMM_OK;
  char buf[96];
  std::snprintf(buf, sizeof buf, "dtype code %d is none of f16 (0), bf16 (1), f32 (6)", dtype);
  return fail(GEMM_ERR_UNSUPPORTED, buf);
}

// Y = op(A) @ op(B) + R, one of the products that another operator is made of: the
// checks and the kernel choice of gemm_linear (without GEMM_LAYER_TILE, which names
// a kernel for a call's own product), and the launch if wanted. Defined in
// layer_api.hip.
struct DenseCall {
  int64_t M, N, K;
  int dtype;
  bool ta, tb;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  const void* R;  // null: none
  int64_t ldr;
  void* Y;
  int64_t ldy;
  int out_dtype;
  const float* scale;  // a factor of the product on the GPU; null: none
};
int run_dense(const DenseCall& c, bool launch, hipStream_t s);

// The same of gemm_grouped_grad_weight: D_g = A_g^T @ B_g (+ D_g).
struct SumsCall {
  int64_t G, M, N, K;
  int dtype;
  const int32_t* offsets;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  void* D;
  int64_t ldd, stride_d;
  int out_dtype;
  bool accumulate;
  const float* scale;  // as above
};
int run_sums(const SumsCall& c, bool launch, hipStream_t s);

}  // namespace dgt
