// Host-side interface of the 8-bit operators: quantisation to e4m3 with a
// scale for each 128 elements (or 128 x 128 block), and the grouped product of
// two such operands.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int F8_GROUP = 128;     // elements of K under one scale
constexpr int kFp8MaxGroups = 256;

// ------------------------------------------------------------ quantisation
struct QuantFp8Args {
  const void* x;        // [G][R][K], rows ldx elements apart, matrices gsx = R ldx
  int x_is_bf16;
  int G, R, K;
  int64_t ldx, gsx;
  int block_rows;       // rows under one scale: 1 or 128
  int transpose;        // codes and scales of the transposed matrices [K][R]
  uint8_t* codes;       // [G][R or K], rows ldc bytes apart, matrices one after another (gsc bytes)
  int64_t ldc, gsc;
  float* scales;        // rows lds floats apart, matrices one after another (gss floats)
  int64_t lds, gss;
};
cudaError_t launch_quantize_fp8(const QuantFp8Args& a, cudaStream_t s);

// ------------------------------------------------------------ products
// FP8_BF16 / FP8_F32: the product itself; FP8_F32 with row_gate scales row r
// by row_gate[r], and with ksplit > 1 writes one partial per K range.
// FP8_SWIGLU / FP8_RELU: the activation of the product(s), quantised to e4m3
// with a scale for each 128 columns of a row.
// FP8_PAIR_F32: the two products of a SwiGLU layer as they are, W3's
// pair_stride elements behind W1's (one partial per K range).
// FP8_GATE_H16: row_gate times the product in fp16, each 128 columns of a row
// by a power of two that takes their largest to [2^14, 2^15); out_scales holds
// its inverse.  (Groups of over 64 rows at most, so of whole tiles.)
enum Fp8Epi { FP8_BF16 = 0, FP8_F32 = 1, FP8_SWIGLU = 2, FP8_RELU = 3, FP8_PAIR_F32 = 4, FP8_GATE_H16 = 5 };

struct Fp8Args {
  int epi;
  int G, N, K;
  int64_t a_rows;          // rows of A (and of the output)
  int64_t max_group_rows;  // no group has more rows
  const uint8_t* A;        // [a_rows][K] codes, rows lda bytes apart
  int64_t lda;
  const float* sa;         // scale of (row, k-block): sa[row * sa_ld + kb]
  int64_t sa_ld;
  const uint8_t* B0;       // [G][N][K] codes, rows ldb bytes apart (W1 or W2), matrices gsb apart
  const uint8_t* B1;       // W3 (FP8_SWIGLU)
  int64_t ldb, gsb;
  const float* sb0;        // scales [G][N or ceil(N / 128)][ceil(K / 128)]
  const float* sb1;
  int b_rows;              // rows of B under one scale: 128 or 1
  void* out;               // bf16 / fp32 [a_rows][N], rows ld_out elements apart; codes for the activations
  int64_t ld_out;
  float* out_scales;       // activations, FP8_GATE_H16: [a_rows][ceil(N / 128)]
  int ksplit;
  int cluster;             // > 1: K ranges summed within a cluster of CTAs (fp8_cluster), no partials
  int64_t split_stride;    // elements between the partials of consecutive K ranges
  int64_t pair_stride;     // FP8_PAIR_F32
  const float* row_gate;   // FP8_F32: may be NULL
  const int32_t* offsets;  // [G + 1] first row of each group; NULL: one group of all rows
  unsigned int* err;
};

struct Fp8Params {
  int G, N, n_tiles, num_kb, ksplit, kb_per, cluster;
  int64_t a_rows;
  const float* sa;
  int64_t sa_ld;
  const float *sb0, *sb1;
  int64_t sb_gs;           // floats between the scales of consecutive groups
  void* out;
  int64_t ld_out, split_stride, pair_stride;
  float* out_scales;
  int vec_out;             // output rows can be written 16 bytes at a time
  int tma_out;             // and whole tiles by TMA
  const float* row_gate;
  const int32_t* offsets;
  unsigned int* err;
  uint64_t limit_ns;
};

struct Fp8Plan {
  CUtensorMap a, b0, b1, out;
  Fp8Params p;
  int epi, ar, sb1;
};

// K ranges of a product with at most `rows` rows over G groups, for one whose
// output tiles alone cannot occupy the GPU.  summed_anyway: its partials cost no
// launch of their own.
int fp8_ksplit(int64_t rows, int G, int N, int K, bool summed_anyway = false);
// The CTAs of a cluster that sum the `ksplit` K ranges of a product among
// themselves; 1: the cut goes through partials and a second launch.
int fp8_cluster(int64_t rows, int ksplit, int K, int b_rows);
cudaError_t plan_fp8(const Fp8Args& g, Fp8Plan* plan, const char** why);
cudaError_t launch_fp8(const Fp8Plan& plan, int num_sms, cudaStream_t s);

// out[r][n] = sum over the ksplit partials (in order) of P[ks][r][n], for the
// rows that belong to a group (offsets NULL: all of them).
struct Fp8ReduceArgs {
  const float* P;
  int ksplit;
  int64_t split_stride, rows;
  int64_t ld;    // floats between rows of a partial, a multiple of 4
  int N;
  void* out;
  int out_is_bf16;
  int64_t ld_out;
  const int32_t* offsets;
  int G;
};
cudaError_t launch_fp8_reduce(const Fp8ReduceArgs& a, cudaStream_t s);

// Codes and scales of the hidden activation of the first *total_rows (at most
// `rows`) rows, from the partials [ksplit] of the first projection (FP8_F32,
// or with pair_stride > 0 FP8_PAIR_F32).
struct Fp8HiddenArgs {
  const float* P;
  int ksplit;
  int64_t split_stride, pair_stride, rows;
  int N;
  const int32_t* total_rows;
  uint8_t* H;   // [rows][N]
  float* Hs;    // [rows][ceil(N / 128)]
};
cudaError_t launch_fp8_hidden(const Fp8HiddenArgs& a, int num_sms, cudaStream_t s);

// y_t = sum over token t's kept choices j (in order) of their rows of Y (fp16,
// times the scale of each 128 columns), then of the shared experts' rows
// *shared_base + s * T + t.  d a multiple of 8.
struct Fp8CombineArgs {
  int64_t T;
  int k, d, n_shared;
  const int32_t* dest_row;     // [T][k], -1: dropped
  const int32_t* shared_base;
  const uint16_t* Y;           // [rows][d]
  const float* scales;         // [rows][ceil(d / 128)]
  void* y;                     // [T][d] bf16
  float* y_f32;                // [T][d] or NULL
};
cudaError_t launch_fp8_combine(const Fp8CombineArgs& a, cudaStream_t s);

}  // namespace moe
