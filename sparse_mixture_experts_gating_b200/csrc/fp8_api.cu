// C ABI of the 8-bit operators: argument checks, workspace and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <string>

#include "moe.h"
#include "fp8.h"
#include "internal.h"

using namespace moe;

namespace {

int fail(int code, const std::string& msg) {
  set_error_message(msg.c_str());
  return code;
}

int done() {
  set_error_message("");
  return MOE_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Floats between the rows of a partial: whole 16-byte pieces.
int64_t partial_ld(int64_t N) { return (N + 3) / 4 * 4; }

// Sizes whose rows, tiles and k-blocks the product counts in 31 bits.
bool product_too_large(int64_t M, int64_t N, int64_t K, int64_t groups) {
  return M > 2147483647LL - 256 || N > (int64_t{1} << 24) || K > (int64_t{1} << 30) ||
         (M / 128 + groups) * ceil_div(N, 128) > 2147483647LL;
}

// How a product's K is cut: into `ranges` whose partials a second launch adds,
// or (ranges 1) among the `cluster` CTAs of a cluster, without partials.
struct Cut {
  int ranges, cluster;
};
Cut cut_of(int64_t M, int64_t N, int64_t K, int64_t groups, int b_rows) {
  const int ks = fp8_ksplit(M, static_cast<int>(groups), static_cast<int>(N), static_cast<int>(K));
  const int cluster = fp8_cluster(M, ks, static_cast<int>(K), b_rows);
  return {cluster > 1 ? 1 : ks, cluster};
}

size_t partial_bytes(int64_t M, int64_t N, int ranges) {
  return ranges > 1 ? sizeof(float) * static_cast<size_t>(ranges) * static_cast<size_t>(M) * static_cast<size_t>(partial_ld(N)) : 0;
}

bool has_plan(int64_t M, int64_t N, int64_t K, int64_t groups) {
  return M > 0 && N > 0 && K > 0 && groups > 0 && groups <= kFp8MaxGroups && !product_too_large(M, N, K, groups);
}

int quantize_fp8(const void* x, int dtype, int64_t matrices, int64_t rows, int64_t K, int64_t ld, int block_rows,
                     int transpose, void* codes, int64_t ld_codes, float* scales, void* stream) {
  const std::string F = "moe_quantize_fp8: ";
  if (matrices < 0 || rows < 0 || K < 0) return fail(MOE_ERR_INVALID_ARG, F + "matrices, rows or K < 0");
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, F + "unknown dtype");
  if (block_rows != 1 && block_rows != F8_GROUP) return fail(MOE_ERR_INVALID_ARG, F + "block_rows must be 1 or 128");
  if (matrices == 0 || rows == 0 || K == 0) return done();
  const int64_t out_rows = transpose ? K : rows, out_cols = transpose ? rows : K;
  if (ld < K || ld_codes < out_cols) return fail(MOE_ERR_INVALID_ARG, F + "a row stride is smaller than its row");
  if (rows > (int64_t{1} << 30) || K > (int64_t{1} << 30) || ld > (int64_t{1} << 32) || ld_codes > (int64_t{1} << 32))
    return fail(MOE_ERR_UNSUPPORTED, F + "rows, K or a row stride is too large");
  // groups (or tiles) are counted in 31 bits
  const int64_t per = block_rows == 1 && !transpose ? rows * ceil_div(K, F8_GROUP)
                                                    : ceil_div(rows, F8_GROUP) * ceil_div(K, F8_GROUP);
  if (matrices > 2147483647LL || per > 2147483647LL / matrices)
    return fail(MOE_ERR_UNSUPPORTED, F + "too many groups of 128 elements");
  if (x == nullptr || codes == nullptr || scales == nullptr) return fail(MOE_ERR_INVALID_ARG, F + "NULL pointer");
  if (!aligned(x, dtype == MOE_BF16 ? 2 : 4) || !aligned(scales, 4))
    return fail(MOE_ERR_INVALID_ARG, F + "x must be aligned to its elements and scales to 4 bytes");
  QuantFp8Args a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.x_is_bf16 = dtype == MOE_BF16;
  a.G = static_cast<int>(matrices);
  a.R = static_cast<int>(rows);
  a.K = static_cast<int>(K);
  a.ldx = ld;
  a.gsx = rows * ld;
  a.block_rows = block_rows;
  a.transpose = transpose != 0;
  a.codes = static_cast<uint8_t*>(codes);
  a.ldc = ld_codes;
  a.gsc = out_rows * ld_codes;
  a.scales = scales;
  a.lds = ceil_div(out_cols, F8_GROUP);
  a.gss = ceil_div(out_rows, block_rows) * a.lds;
  const cudaError_t e = launch_quantize_fp8(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, F + cudaGetErrorString(e));
  return done();
}

int matmul_fp8(int64_t M, int64_t N, int64_t K, int64_t groups, const void* a_codes, int64_t lda, const float* a_scales,
               const void* b_codes, int64_t ldb, const float* b_scales, int b_rows, const int32_t* offsets, void* out,
               int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream) {
  const std::string F = "moe_matmul_fp8: ";
  if (M < 0 || N < 1 || K < 1) return fail(MOE_ERR_INVALID_ARG, F + "need M >= 0, N >= 1 and K >= 1");
  if (groups < 1 || groups > kFp8MaxGroups) return fail(MOE_ERR_INVALID_ARG, F + "groups must be in [1, 256]");
  if (groups > 1 && offsets == nullptr) return fail(MOE_ERR_INVALID_ARG, F + "several groups need their offsets");
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, F + "unknown out_dtype");
  if (b_rows != 1 && b_rows != F8_GROUP) return fail(MOE_ERR_INVALID_ARG, F + "b_rows must be 1 or 128");
  if (M == 0) return done();
  if (product_too_large(M, N, K, groups)) return fail(MOE_ERR_UNSUPPORTED, F + "a size is too large");
  if (lda >= (int64_t{1} << 40) || ldb >= (int64_t{1} << 40) || ldb > ((int64_t{1} << 40) - 1) / N ||
      ld_out > (int64_t{1} << 60) / M)
    return fail(MOE_ERR_UNSUPPORTED, F + "a row stride is too large");
  if (lda < K || ldb < K || ld_out < N) return fail(MOE_ERR_INVALID_ARG, F + "a row stride is smaller than its row");
  if (a_codes == nullptr || a_scales == nullptr || b_codes == nullptr || b_scales == nullptr || out == nullptr)
    return fail(MOE_ERR_INVALID_ARG, F + "NULL pointer");
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || lda % 16 != 0 || ldb % 16 != 0)
    return fail(MOE_ERR_INVALID_ARG, F + "codes and their row strides must be multiples of 16 bytes");
  if (!aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(offsets, 4) || !aligned(out, out_dtype == MOE_BF16 ? 2 : 4))
    return fail(MOE_ERR_INVALID_ARG, F + "scales, offsets and out must be aligned to their elements");
  const Cut cut = cut_of(M, N, K, groups, b_rows);
  const size_t need = partial_bytes(M, N, cut.ranges);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256)))
    return fail(MOE_ERR_INVALID_ARG, F + "workspace missing, not 256-byte aligned or smaller than "
                                         "moe_matmul_fp8_scratch_bytes()");
  int num_sms = 0;
  unsigned int* err = nullptr;
  cudaError_t e = current_device_info(&num_sms, &err);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, F + cudaGetErrorString(e));
  const int ks = cut.ranges;
  Fp8Args a;
  memset(&a, 0, sizeof(a));
  a.epi = ks > 1 || out_dtype == MOE_F32 ? FP8_F32 : FP8_BF16;
  a.G = static_cast<int>(groups);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.a_rows = M;
  a.max_group_rows = M;
  a.A = static_cast<const uint8_t*>(a_codes);
  a.lda = lda;
  a.sa = a_scales;
  a.sa_ld = ceil_div(K, F8_GROUP);
  a.B0 = static_cast<const uint8_t*>(b_codes);
  a.ldb = ldb;
  a.gsb = ldb * N;
  a.sb0 = b_scales;
  a.b_rows = b_rows;
  a.out = ks > 1 ? workspace : out;
  a.ld_out = ks > 1 ? partial_ld(N) : ld_out;
  a.ksplit = ks;
  a.cluster = cut.cluster;
  a.split_stride = ks > 1 ? M * partial_ld(N) : 0;
  a.offsets = offsets;
  a.err = err;
  Fp8Plan plan;
  const char* why = nullptr;
  if (plan_fp8(a, &plan, &why) != cudaSuccess) return fail(MOE_ERR_UNSUPPORTED, F + (why ? why : "plan failed"));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = launch_fp8(plan, num_sms, s);
  if (e == cudaSuccess && ks > 1) {
    Fp8ReduceArgs r;
    memset(&r, 0, sizeof(r));
    r.P = static_cast<const float*>(workspace);
    r.ksplit = ks;
    r.split_stride = M * partial_ld(N);
    r.ld = partial_ld(N);
    r.rows = M;
    r.N = static_cast<int>(N);
    r.out = out;
    r.out_is_bf16 = out_dtype == MOE_BF16;
    r.ld_out = ld_out;
    r.offsets = offsets;
    r.G = static_cast<int>(groups);
    e = launch_fp8_reduce(r, s);
  }
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, F + cudaGetErrorString(e));
  return done();
}
}  // namespace

// No C++ exception (a message that finds no memory) leaves a C entry.
extern "C" {

int moe_quantize_fp8(const void* x, int dtype, int64_t matrices, int64_t rows, int64_t K, int64_t ld, int block_rows,
                     int transpose, void* codes, int64_t ld_codes, float* scales, void* stream) {
  try {
    return quantize_fp8(x, dtype, matrices, rows, K, ld, block_rows, transpose, codes, ld_codes, scales, stream);
  } catch (...) {
    return MOE_ERR_CUDA;
  }
}

size_t moe_matmul_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t groups) {
  return moe_matmul_fp8_scratch_bytes(M, N, K, groups, 1);  // (never summed in clusters)
}

size_t moe_matmul_fp8_scratch_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, int b_rows) {
  if (!has_plan(M, N, K, groups) || (b_rows != 1 && b_rows != F8_GROUP)) return 0;
  return partial_bytes(M, N, cut_of(M, N, K, groups, b_rows).ranges);
}

int moe_matmul_fp8(int64_t M, int64_t N, int64_t K, int64_t groups, const void* a_codes, int64_t lda,
                   const float* a_scales, const void* b_codes, int64_t ldb, const float* b_scales, int b_rows,
                   const int32_t* offsets, void* out, int out_dtype, int64_t ld_out, void* workspace,
                   size_t workspace_bytes, void* stream) {
  try {
    return matmul_fp8(M, N, K, groups, a_codes, lda, a_scales, b_codes, ldb, b_scales, b_rows, offsets, out, out_dtype,
                      ld_out, workspace, workspace_bytes, stream);
  } catch (...) {
    return MOE_ERR_CUDA;
  }
}

}  // extern "C"
