// Host-side interface of the router's balance loss of each sequence.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kBalanceMaxE = 256;

struct BalanceArgs {
  int64_t T, B;
  int E, k;
  const void* logits;       // [T][E]
  int is_bf16;
  int sigmoid;              // scores: softmax (0) or normalised sigmoid (1)
  const int32_t* offsets;   // [B + 1]; NULL: one sequence of T tokens
  const uint8_t* mask;      // [T], 0: padding; NULL: none
  // forward
  float *aux, *z;           // [B]
  int32_t *counts, *tokens; // [B][E], [B]
  void* workspace;
  int tile;                 // tokens per tile
  int64_t tiles;
  // backward
  const int32_t *counts_in, *tokens_in;
  const float *daux, *dz;   // [B], either may be NULL
  float* dlogits;           // [T][E]
};

// Tokens per tile of a batch of T tokens, and the bytes of the tiles' partials.
int balance_tile(int64_t T);
size_t balance_workspace_bytes(int64_t T, int E, int64_t B);
cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s);
cudaError_t launch_balance_backward(const BalanceArgs& a, cudaStream_t s);

}  // namespace moe
