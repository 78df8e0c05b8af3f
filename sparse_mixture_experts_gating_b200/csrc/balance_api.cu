// C ABI of the router's balance loss: argument checks, workspace and launches.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <string>

#include "moe.h"
#include "balance.h"
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

// Tokens are counted in 31 bits, with room for a thread's steps past the last one.
constexpr int64_t kMaxCount = 2147483647LL - 256;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The checks that both directions share; fills the common arguments.
int common(const std::string& F, int64_t T, int E, int k, const void* logits, int dtype, int scoring, int64_t sequences,
           const int32_t* offsets, const uint8_t* mask, BalanceArgs* a) {
  if (T < 0 || sequences < 0) return fail(MOE_ERR_INVALID_ARG, F + "T or sequences < 0");
  if (E < 1 || E > kBalanceMaxE) return fail(MOE_ERR_INVALID_ARG, F + "num_experts must be in [1, 256]");
  if (k < 1 || k > E || k > 8) return fail(MOE_ERR_INVALID_ARG, F + "need 1 <= k <= min(E, 8)");
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, F + "unknown dtype");
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARG, F + "unknown scoring");
  if (offsets == nullptr && sequences != 1) return fail(MOE_ERR_INVALID_ARG, F + "several sequences need their offsets");
  if (T > kMaxCount || sequences > kMaxCount) return fail(MOE_ERR_UNSUPPORTED, F + "T or sequences too large");
  if (T > 0 && logits == nullptr) return fail(MOE_ERR_INVALID_ARG, F + "logits is NULL");
  if (!aligned(logits, dtype == MOE_BF16 ? 2 : 4) || !aligned(offsets, 4))
    return fail(MOE_ERR_INVALID_ARG, F + "logits and offsets must be aligned to their elements");
  memset(a, 0, sizeof(*a));
  a->T = T;
  a->B = sequences;
  a->E = E;
  a->k = k;
  a->logits = logits;
  a->is_bf16 = dtype == MOE_BF16;
  a->sigmoid = scoring == MOE_SCORE_SIGMOID;
  a->offsets = offsets;
  a->mask = mask;
  return MOE_OK;
}

int router_balance(int64_t T, int num_experts, int k, const void* logits, int dtype, int scoring, int64_t sequences,
                       const int32_t* offsets, const uint8_t* mask, float* aux, float* z, int32_t* counts,
                       int32_t* tokens, void* workspace, size_t workspace_bytes, void* stream) {
  const std::string F = "moe_router_balance: ";
  BalanceArgs a;
  const int rc = common(F, T, num_experts, k, logits, dtype, scoring, sequences, offsets, mask, &a);
  if (rc != MOE_OK) return rc;
  if (sequences == 0) return done();
  if (aux == nullptr || z == nullptr || counts == nullptr || tokens == nullptr)
    return fail(MOE_ERR_INVALID_ARG, F + "an output pointer is NULL");
  if (!aligned(aux, 4) || !aligned(z, 4) || !aligned(counts, 4) || !aligned(tokens, 4))
    return fail(MOE_ERR_INVALID_ARG, F + "outputs must be aligned to their elements");
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < balance_workspace_bytes(T, num_experts, sequences))
    return fail(MOE_ERR_INVALID_ARG, F + "workspace missing, not 16-byte aligned or smaller than "
                                         "moe_router_balance_workspace_bytes()");
  a.aux = aux;
  a.z = z;
  a.counts = counts;
  a.tokens = tokens;
  a.workspace = workspace;
  a.tile = balance_tile(T);
  a.tiles = (T + a.tile - 1) / a.tile;
  const cudaError_t e = launch_balance(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, F + cudaGetErrorString(e));
  return done();
}

int router_balance_backward(int64_t T, int num_experts, int k, const void* logits, int dtype, int scoring,
                                int64_t sequences, const int32_t* offsets, const uint8_t* mask, const int32_t* counts,
                                const int32_t* tokens, const float* daux, const float* dz, float* dlogits,
                                void* stream) {
  const std::string F = "moe_router_balance_backward: ";
  BalanceArgs a;
  const int rc = common(F, T, num_experts, k, logits, dtype, scoring, sequences, offsets, mask, &a);
  if (rc != MOE_OK) return rc;
  if (T == 0) return done();
  if (dlogits == nullptr || (sequences > 0 && (counts == nullptr || tokens == nullptr)))
    return fail(MOE_ERR_INVALID_ARG, F + "dlogits, counts and tokens must be non-NULL");
  if (!aligned(dlogits, 4) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(daux, 4) || !aligned(dz, 4))
    return fail(MOE_ERR_INVALID_ARG, F + "counts, tokens and gradients must be aligned to their elements");
  cudaError_t e;
  if (sequences == 0) {
    e = cudaMemsetAsync(dlogits, 0, sizeof(float) * static_cast<size_t>(T) * num_experts, static_cast<cudaStream_t>(stream));
  } else {
    a.counts_in = counts;
    a.tokens_in = tokens;
    a.daux = daux;
    a.dz = dz;
    a.dlogits = dlogits;
    e = launch_balance_backward(a, static_cast<cudaStream_t>(stream));
  }
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, F + cudaGetErrorString(e));
  return done();
}

}  // namespace

// No C++ exception (a message that finds no memory) leaves a C entry.
extern "C" {

size_t moe_router_balance_workspace_bytes(int64_t T, int num_experts, int64_t sequences) {
  if (T < 0 || num_experts < 1 || num_experts > kBalanceMaxE || sequences < 0 || T > kMaxCount || sequences > kMaxCount)
    return 0;
  return balance_workspace_bytes(T, num_experts, sequences);
}

int moe_router_balance(int64_t T, int num_experts, int k, const void* logits, int dtype, int scoring, int64_t sequences,
                       const int32_t* offsets, const uint8_t* mask, float* aux, float* z, int32_t* counts,
                       int32_t* tokens, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    return router_balance(T, num_experts, k, logits, dtype, scoring, sequences, offsets, mask, aux, z, counts, tokens,
                          workspace, workspace_bytes, stream);
  } catch (...) {
    return MOE_ERR_CUDA;
  }
}

int moe_router_balance_backward(int64_t T, int num_experts, int k, const void* logits, int dtype, int scoring,
                                int64_t sequences, const int32_t* offsets, const uint8_t* mask, const int32_t* counts,
                                const int32_t* tokens, const float* daux, const float* dz, float* dlogits,
                                void* stream) {
  try {
    return router_balance_backward(T, num_experts, k, logits, dtype, scoring, sequences, offsets, mask, counts, tokens,
                                   daux, dz, dlogits, stream);
  } catch (...) {
    return MOE_ERR_CUDA;
  }
}

}  // extern "C"
