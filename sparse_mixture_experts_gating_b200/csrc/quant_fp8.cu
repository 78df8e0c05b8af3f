// Quantisation to 8-bit floating point (e4m3) with a scale for each group of
// 128 elements of a row, or for each 128 x 128 block.
//
// For a block with largest magnitude m:  a = max(m, 2^-100),
//   scale = fl(a / 448),  code = e4m3(fl(x * fl(448 / a)))
// with fl the rounding to fp32 and e4m3 the rounding to the nearest code (ties
// to even).  Each step is one IEEE operation, so codes and scales do not
// depend on how the work is split.  a > 0 keeps an all-zero block at codes 0
// without a special case; 448 / a stays finite down to a = 2^-100.  A NaN
// keeps the NaN code; an infinity makes its block's scale infinite, so that
// the whole block reads back as NaN.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "internal.h"

namespace moe {
namespace {

// Eight consecutive elements of a row from column c on, as fp32; columns past
// K read as 0.  vec: the row's 16-byte pieces are aligned and c + 8 <= K.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int c, int K, bool vec, float (&v)[8]) {
  if (vec && c + 8 <= K) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + c));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < K ? __bfloat162float(p[c + i]) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* p, int c, int K, bool vec, float (&v)[8]) {
  if (vec && c + 8 <= K) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + c));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p + c + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < K ? p[c + i] : 0.f;
  }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// n <= 8 bytes of `c` to dst; vec: dst is 8-byte aligned.
__device__ __forceinline__ void store8(uint8_t* dst, uint2 c, int n, bool vec) {
  if (vec && n >= 8) {
    *reinterpret_cast<uint2*>(dst) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) dst[i] = static_cast<uint8_t>(i < 4 ? c.x >> (8 * i) : c.y >> (8 * (i - 4)));
  }
}

// Groups of 128 elements of a row: 16 lanes per group, 8 elements per lane.
// Grid-stride over the R * ceil(K / 128) groups of every matrix.
template <typename XT>
__global__ void __launch_bounds__(256) quant_rows_kernel(const QuantFp8Args a, int kb_n, int vec_in, int vec_out) {
  const int l = threadIdx.x & 15;
  const int64_t teams = static_cast<int64_t>(gridDim.x) * 16;
  const int64_t items = static_cast<int64_t>(a.G) * a.R * kb_n;
  const XT* x = static_cast<const XT*>(a.x);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  // every lane of a warp runs the same number of steps: the shuffles below need both its teams
  for (int64_t i0 = first & ~int64_t{1}; i0 < items; i0 += teams) {
    const int64_t i = i0 + (first & 1);
    const bool live = i < items;
    const uint32_t ii = live ? static_cast<uint32_t>(i) : 0u;
    const uint32_t row = ii / static_cast<uint32_t>(kb_n);
    const int g = static_cast<int>(ii - row * static_cast<uint32_t>(kb_n));
    const uint32_t mat = row / static_cast<uint32_t>(a.R), r = row - mat * static_cast<uint32_t>(a.R);
    const int c = g * F8_GROUP + l * 8;
    float v[8];
    load8(x + static_cast<int64_t>(mat) * a.gsx + static_cast<int64_t>(r) * a.ldx, c, live ? a.K : 0, vec_in, v);
    float m = amax8(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const Fp8Scale q = fp8_scale(m);
    if (live) {
      uint8_t* dst = a.codes + static_cast<int64_t>(mat) * a.gsc + static_cast<int64_t>(r) * a.ldc + c;
      store8(dst, codes8(v, q.inv), a.K - c, vec_out);
      if (l == 0) a.scales[static_cast<int64_t>(mat) * a.gss + static_cast<int64_t>(r) * a.lds + g] = q.scale;
    }
  }
}

// One 128 x 128 tile of a matrix per CTA: thread (ty, tx) holds rows ty + 16 j
// and columns 8 tx .. 8 tx + 7.  BLOCK: one scale for the tile; else (the
// transposed matrix in groups along its rows) one for each column of the tile.
template <typename XT, bool BLOCK, bool TR>
__global__ void __launch_bounds__(256) quant_tile_kernel(const QuantFp8Args a, int rb_n, int kb_n, int vec_in,
                                                         int vec_out) {
  static_assert(BLOCK || TR, "rows of an untransposed matrix take the row kernel");
  __shared__ float s_red[BLOCK ? 8 : 16 * 128];
  __shared__ alignas(16) uint8_t s_t[TR ? 128 * 144 : 16];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const uint32_t per = static_cast<uint32_t>(rb_n) * static_cast<uint32_t>(kb_n);
  const uint32_t mat = blockIdx.x / per, tile = blockIdx.x - mat * per;
  const int rb = static_cast<int>(tile / static_cast<uint32_t>(kb_n));
  const int kb = static_cast<int>(tile - static_cast<uint32_t>(rb) * static_cast<uint32_t>(kb_n));
  const XT* x = static_cast<const XT*>(a.x) + static_cast<int64_t>(mat) * a.gsx;
  const int c = kb * 128 + tx * 8;
  float v[8][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = rb * 128 + ty + 16 * j;
    load8(x + static_cast<int64_t>(r) * a.ldx, c, r < a.R ? a.K : 0, vec_in, v[j]);
  }
  float inv[8];
  if (BLOCK) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, amax8(v[j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, s_red[i]);
    const Fp8Scale q = fp8_scale(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) inv[i] = q.inv;
    if (threadIdx.x == 0)
      a.scales[static_cast<int64_t>(mat) * a.gss + (TR ? kb * a.lds + rb : rb * a.lds + kb)] = q.scale;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = fabsf(v[0][i]);
#pragma unroll
      for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(v[j][i]));
      s_red[ty * 128 + tx * 8 + i] = m;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = s_red[tx * 8 + i];
#pragma unroll
      for (int t = 1; t < 16; ++t) m = fmaxf(m, s_red[t * 128 + tx * 8 + i]);
      const Fp8Scale q = fp8_scale(m);
      inv[i] = q.inv;
      if (ty == 0 && c + i < a.K) a.scales[static_cast<int64_t>(mat) * a.gss + static_cast<int64_t>(c + i) * a.lds + rb] = q.scale;
    }
  }
  uint8_t* codes = a.codes + static_cast<int64_t>(mat) * a.gsc;
  if (!TR) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = rb * 128 + ty + 16 * j;
      if (r < a.R) store8(codes + static_cast<int64_t>(r) * a.ldc + c, codes8(v[j], inv[0]), a.K - c, vec_out);
    }
  } else {
    // through shared memory: row k of the tile's transpose, 144 bytes apart
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t w = e4m3x2(v[j][i] * inv[i], v[j + 1][i] * inv[i]);
        s_t[(tx * 8 + i) * 144 + ty + 16 * j] = static_cast<uint8_t>(w);
        s_t[(tx * 8 + i) * 144 + ty + 16 * (j + 1)] = static_cast<uint8_t>(w >> 8);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = ty + 16 * j, r = rb * 128 + tx * 8;
      if (kb * 128 + k < a.K)
        store8(codes + static_cast<int64_t>(kb * 128 + k) * a.ldc + r, *reinterpret_cast<const uint2*>(s_t + k * 144 + tx * 8),
               a.R - r, vec_out);
    }
  }
}

template <typename XT>
cudaError_t launch_x(const QuantFp8Args& a, cudaStream_t s) {
  const int elt = static_cast<int>(sizeof(XT));
  const int kb = (a.K + 127) / 128, rb = (a.R + 127) / 128;
  const int vec_in = ((reinterpret_cast<uintptr_t>(a.x) | static_cast<uintptr_t>(a.ldx * elt) |
                       static_cast<uintptr_t>(a.gsx * elt)) & 15) == 0;
  const int vec_out = ((reinterpret_cast<uintptr_t>(a.codes) | static_cast<uintptr_t>(a.ldc) |
                        static_cast<uintptr_t>(a.gsc)) & 7) == 0;
  if (a.block_rows == 1 && !a.transpose) {
    const int64_t items = static_cast<int64_t>(a.G) * a.R * kb;
    int64_t blocks = (items + 15) / 16;
    if (blocks > 148 * 16) blocks = 148 * 16;
    quant_rows_kernel<XT><<<static_cast<unsigned>(blocks), 256, 0, s>>>(a, kb, vec_in, vec_out);
  } else {
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.G) * rb * kb);
    if (a.block_rows == 128) {
      if (a.transpose) quant_tile_kernel<XT, true, true><<<blocks, 256, 0, s>>>(a, rb, kb, vec_in, vec_out);
      else quant_tile_kernel<XT, true, false><<<blocks, 256, 0, s>>>(a, rb, kb, vec_in, vec_out);
    } else {
      quant_tile_kernel<XT, false, true><<<blocks, 256, 0, s>>>(a, rb, kb, vec_in, vec_out);
    }
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_fp8(const QuantFp8Args& a, cudaStream_t s) {
  if (a.G == 0 || a.R == 0 || a.K == 0) return cudaSuccess;
  return a.x_is_bf16 ? launch_x<__nv_bfloat16>(a, s) : launch_x<float>(a, s);
}

}  // namespace moe
