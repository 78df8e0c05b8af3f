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
//
// What bounds it: HBM.  bf16, 8192 x 4096: rows 19.5 us (5.2 TB/s, 2 us of it the
// launch), transposed rows 22.9 us, transposed blocks 18.7 us; 128 x 768 x 2048 in
// blocks 96 us (6.4 TB/s); fp32, 8192 x 4096: rows 26.0 us (6.5 TB/s).  Rows whose
// 16-byte pieces are not aligned (8192 x 4093 bf16) are loaded element by element:
// rows 31.3 us, transposed rows 42.3 us, blocks 36.7 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "internal.h"

namespace moe {
namespace {

// Eight consecutive elements of a row, as they are loaded.
template <typename XT>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  __device__ __forceinline__ float amax() const {  // (exact on pairs: a maximum rounds nothing)
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    __nv_bfloat162 m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    m[0] = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
    return fmaxf(__low2float(m[0]), __high2float(m[0]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ float at(int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
  __device__ __forceinline__ float amax() const {
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                 fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
  }
};

// Elements c .. c + 7 of row p; columns past K read as 0.  vec: the row's
// 16-byte pieces are aligned.
__device__ __forceinline__ Eight<__nv_bfloat16> load8(const __nv_bfloat16* p, int c, int K, bool vec) {
  Eight<__nv_bfloat16> v;
  if (vec && c + 8 <= K) {
    v.u = __ldg(reinterpret_cast<const uint4*>(p + c));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = c + 2 * i < K ? __bfloat16_as_ushort(p[c + 2 * i]) : 0u;
      const uint32_t hi = c + 2 * i + 1 < K ? __bfloat16_as_ushort(p[c + 2 * i + 1]) : 0u;
      w[i] = lo | hi << 16;
    }
    v.u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}
__device__ __forceinline__ Eight<float> load8(const float* p, int c, int K, bool vec) {
  Eight<float> v;
  if (vec && c + 8 <= K) {
    v.a = __ldg(reinterpret_cast<const float4*>(p + c));
    v.b = __ldg(reinterpret_cast<const float4*>(p + c + 4));
  } else {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = c + i < K ? p[c + i] : 0.f;
    v.a = make_float4(w[0], w[1], w[2], w[3]);
    v.b = make_float4(w[4], w[5], w[6], w[7]);
  }
  return v;
}

template <typename XT>
__device__ __forceinline__ uint2 codes8(const Eight<XT>& v, float inv) {
  return make_uint2(e4m3x4(v.at(0) * inv, v.at(1) * inv, v.at(2) * inv, v.at(3) * inv),
                    e4m3x4(v.at(4) * inv, v.at(5) * inv, v.at(6) * inv, v.at(7) * inv));
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

// Groups of 128 elements of a row: 16 lanes per group, 8 elements per lane,
// UNROLL groups of a team of 16 lanes in flight at once (one load of 16 bytes
// per lane keeps 32 KB in flight per SM, too few for HBM's latency).  A block
// takes 16 x UNROLL consecutive groups.
constexpr int UNROLL = 4;

template <typename XT>
__global__ void __launch_bounds__(256) quant_rows_kernel(const QuantFp8Args a, uint32_t rows, int kb_n, int step_rows,
                                                         int step_groups, int vec_in, int vec_out) {
  static_assert(UNROLL == 4, "a lane divides for one group in four");
  const int l = threadIdx.x & 15;
  pdl_wait();
  pdl_trigger();
  // this team's first group; the next ones lie 16 groups = step_rows rows and step_groups groups on
  const uint32_t i0 = blockIdx.x * (16u * UNROLL) + (threadIdx.x >> 4);
  uint32_t r = i0 / static_cast<uint32_t>(kb_n);
  int g = static_cast<int>(i0 - r * static_cast<uint32_t>(kb_n));
  // every lane runs every step: the shuffles need both teams of a warp
  Eight<XT> v[UNROLL];
  uint8_t* dst[UNROLL];
  int left[UNROLL];  // elements from this lane's first one to the end of the row; 0 or less: none
  uint32_t my_row = 0;  // of the group that this lane divides for
  int my_g = 0;
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const bool live = r < rows;
    const int c = g * F8_GROUP + l * 8;
    left[u] = live ? a.K - c : 0;
    dst[u] = a.codes + static_cast<int64_t>(r) * a.ldc + c;
    v[u] = load8(static_cast<const XT*>(a.x) + static_cast<int64_t>(live ? r : 0u) * a.ldx, c, live ? a.K : 0, vec_in);
    if ((l & 3) == u) {
      my_row = r;
      my_g = g;
    }
    r += static_cast<uint32_t>(step_rows);
    g += step_groups;
    if (g >= kb_n) {
      g -= kb_n;
      ++r;
    }
  }
  float m[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) m[u] = v[u].amax();
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
  // two divisions a lane, not eight: lane l of a team divides for group l & 3
  const Fp8Scale q = fp8_scale((l & 2) ? ((l & 1) ? m[3] : m[2]) : ((l & 1) ? m[1] : m[0]));
  if (l < UNROLL && my_row < rows) a.scales[static_cast<int64_t>(my_row) * a.lds + my_g] = q.scale;
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const float inv = __shfl_sync(0xffffffffu, q.inv, (threadIdx.x & 16) + u);
    store8(dst[u], codes8(v[u], inv), left[u], vec_out);
  }
}

// One 128 x 128 tile of a matrix per CTA: thread (ty, tx) holds rows 8 ty .. 8 ty
// + 7 and columns 8 tx .. 8 tx + 7.  BLOCK: one scale for the tile; else (the
// transposed matrix in groups along its rows) one for each column of the tile.
// TR: the codes go out transposed, through shared memory in units of 8 bytes
// (8 rows of a column), unit u of column k at u ^ (k / 8) of the column's 128
// bytes, so that neither side meets a bank twice.
template <typename XT, bool BLOCK, bool TR>
__global__ void __launch_bounds__(256) quant_tile_kernel(const QuantFp8Args a, int rb_n, int kb_n, int vec_in,
                                                         int vec_out) {
  static_assert(BLOCK || TR, "rows of an untransposed matrix take the row kernel");
  __shared__ alignas(16) float s_red[BLOCK ? 8 : 8 * 128];
  __shared__ alignas(16) float s_inv[BLOCK ? 4 : 128];
  __shared__ alignas(16) uint8_t s_t[TR ? 128 * 128 : 16];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const uint32_t per = static_cast<uint32_t>(rb_n) * static_cast<uint32_t>(kb_n);
  pdl_wait();
  pdl_trigger();
  const uint32_t mat = blockIdx.x / per, tile = blockIdx.x - mat * per;
  const int rb = static_cast<int>(tile / static_cast<uint32_t>(kb_n));
  const int kb = static_cast<int>(tile - static_cast<uint32_t>(rb) * static_cast<uint32_t>(kb_n));
  const XT* x = static_cast<const XT*>(a.x) + static_cast<int64_t>(mat) * a.gsx;
  float* scales = a.scales + static_cast<int64_t>(mat) * a.gss;
  const int c = kb * 128 + tx * 8, r0 = rb * 128 + ty * 8;
  Eight<XT> v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = r0 + j;
    v[j] = load8(x + static_cast<int64_t>(r < a.R ? r : 0) * a.ldx, c, r < a.R ? a.K : 0, vec_in);
  }
  float inv[8];
  if (BLOCK) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, v[j].amax());
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) s_red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, s_red[i]);
    const Fp8Scale q = fp8_scale(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) inv[i] = q.inv;
    if (threadIdx.x == 0) scales[TR ? kb * a.lds + rb : rb * a.lds + kb] = q.scale;
  } else {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = fabsf(v[0].at(i));
#pragma unroll
      for (int j = 1; j < 8; ++j) m[i] = fmaxf(m[i], fabsf(v[j].at(i)));
      m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
    }
    if ((threadIdx.x & 16) == 0) {
      float4* red = reinterpret_cast<float4*>(s_red + warp * 128 + tx * 8);
      red[0] = make_float4(m[0], m[1], m[2], m[3]);
      red[1] = make_float4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();
    if (threadIdx.x < 128) {  // a column each
      float t = s_red[threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; ++w) t = fmaxf(t, s_red[w * 128 + threadIdx.x]);
      const Fp8Scale q = fp8_scale(t);
      s_inv[threadIdx.x] = q.inv;
      const int k = kb * 128 + threadIdx.x;
      if (k < a.K) scales[static_cast<int64_t>(k) * a.lds + rb] = q.scale;
    }
    __syncthreads();
    const float4* in = reinterpret_cast<const float4*>(s_inv + tx * 8);
    const float4 lo = in[0], hi = in[1];
    inv[0] = lo.x; inv[1] = lo.y; inv[2] = lo.z; inv[3] = lo.w;
    inv[4] = hi.x; inv[5] = hi.y; inv[6] = hi.z; inv[7] = hi.w;
  }
  uint8_t* codes = a.codes + static_cast<int64_t>(mat) * a.gsc;
  if (!TR) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (r0 + j < a.R) store8(codes + static_cast<int64_t>(r0 + j) * a.ldc + c, codes8(v[j], inv[0]), a.K - c, vec_out);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint2 w = make_uint2(e4m3x4(v[0].at(i) * inv[i], v[1].at(i) * inv[i], v[2].at(i) * inv[i], v[3].at(i) * inv[i]),
                                 e4m3x4(v[4].at(i) * inv[i], v[5].at(i) * inv[i], v[6].at(i) * inv[i], v[7].at(i) * inv[i]));
      *reinterpret_cast<uint2*>(s_t + (tx * 8 + i) * 128 + ((ty ^ tx) << 3)) = w;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = ty + 16 * j, r = rb * 128 + tx * 8;
      if (kb * 128 + k < a.K)
        store8(codes + static_cast<int64_t>(kb * 128 + k) * a.ldc + r,
               *reinterpret_cast<const uint2*>(s_t + k * 128 + ((tx ^ (k >> 3)) << 3)), a.R - r, vec_out);
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
    // (matrices lie one after another, so their rows are rows of one)
    const int64_t rows = static_cast<int64_t>(a.G) * a.R, items = rows * kb;  // below 2^31
    const int64_t blocks = (items + 16 * UNROLL - 1) / (16 * UNROLL);
    return launch_pdl(quant_rows_kernel<XT>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a,
                      static_cast<uint32_t>(rows), kb, 16 / kb, 16 % kb, vec_in, vec_out);
  }
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.G) * rb * kb)), block(256);
  if (a.block_rows != 128) return launch_pdl(quant_tile_kernel<XT, false, true>, grid, block, 0, s, a, rb, kb, vec_in, vec_out);
  return a.transpose ? launch_pdl(quant_tile_kernel<XT, true, true>, grid, block, 0, s, a, rb, kb, vec_in, vec_out)
                     : launch_pdl(quant_tile_kernel<XT, true, false>, grid, block, 0, s, a, rb, kb, vec_in, vec_out);
}

}  // namespace

cudaError_t launch_quantize_fp8(const QuantFp8Args& a, cudaStream_t s) {
  if (a.G == 0 || a.R == 0 || a.K == 0) return cudaSuccess;
  return a.x_is_bf16 ? launch_x<__nv_bfloat16>(a, s) : launch_x<float>(a, s);
}

}  // namespace moe
