// The router's balance loss and z-loss of each sequence of a packed batch,
// with the per-expert counts, and their gradient with respect to the logits.
//
// For the n tokens of a sequence (those that the mask keeps and that have an
// expert left):  c_e = choices of expert e (top-k of the logits, ties to the
// lower index), p_t = softmax(u_t) with u the logits, or log(sigmoid(logits))
// (which is sigmoid normalised over the experts, without its underflow),
//   aux = E / (k n) sum_e c_e (1 / n) sum_t p_te,    z = (1 / n) sum_t lse(l_t)^2.
// The counts have no gradient; with g_e = daux E (c_e - k n / E) / (k n^2)
//   d/dl_te = p_te (g_e - sum_j p_tj g_j) [sigmoid(-l_te)] + dz (2 / n) lse_t softmax(l_t)_e.
// (Taking k n / E off the counts changes nothing, since p sums to 1, and keeps
// the difference from cancelling: counts of a long sequence are all alike.)
//
// W lanes hold one token's logits, J consecutive experts each, so that a
// reduction takes log2(W) shuffles for 32 / W tokens at once.  The forward
// pass sums p and the choices of a tile of tokens in registers, one segment
// (the part of a sequence in the tile) at a time, and writes the segment's
// sums to a slot of its own; a second launch adds each sequence's slots in
// order.  No atomics: results do not depend on timing.
//
// What bounds it: instruction issue, in the choices' shuffles and the
// exponentials.  131072 tokens in 37 sequences, 128 experts, top-4, fp32 (67 MB
// read, in the gradient read and 67 MB written): forward 39 us, gradient 29 us.  In
// one sequence the forward takes 56 us (one CTA adds all 586 tiles' slots), in 4096
// sequences 90 us (every 32 tokens are a segment whose sums are joined and
// written).  A batch of 300 tokens takes its three launches, 12 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "balance.h"
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int THREADS = 256;

// A slot holds psum [E], counts [E], sum of lse^2, tokens.
__host__ __device__ inline int slot_words(int E) { return 2 * E + 2; }

template <int W>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int W>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sequence bounds, clamped into [0, T].
__device__ __forceinline__ int64_t seq_begin(const BalanceArgs& a, int64_t b) {
  if (a.offsets == nullptr) return b == 0 ? 0 : a.T;
  return min(max(static_cast<int64_t>(a.offsets[b]), int64_t{0}), a.T);
}
// The last sequence that begins at or before token t (0 if none does).
__device__ __forceinline__ int64_t seq_of(const BalanceArgs& a, int64_t t) {
  int64_t lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (seq_begin(a, mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// This lane's J logits of a token (experts e0 ..), -inf past E.
template <typename XT, int J>
__device__ __forceinline__ void load_logits(const XT* p, int e0, int E, bool vec, float (&l)[J]) {
  if constexpr (J * sizeof(XT) >= 16) {
    if (vec && e0 + J <= E) {
      constexpr int NV = static_cast<int>(J * sizeof(XT) / 16), PER = 16 / static_cast<int>(sizeof(XT));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + e0) + i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          if constexpr (sizeof(XT) == 4) l[i * PER + j] = __uint_as_float(w[j]);
          else l[i * PER + j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) l[j] = e0 + j < E ? to_f32(p[e0 + j]) : -INFINITY;
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// softmax numerators ex and their sum over the row, of values v with row maximum
// m: exp(v - m) as 2^(v log2 e - m log2 e), one fused operation and one of the
// special function unit.  (The rounding of m log2 e is common to the row, so
// it cancels in the scores, and in m + log of the sum it is as small as m's
// own.)  Beyond |m| = 2^16 that rounding could leave the exponential's range
// (rows of a mask's huge value), and the difference is taken first.
template <int W, int J>
__device__ __forceinline__ float exp_sum(const float (&v)[J], float m, float (&ex)[J]) {
  constexpr float kLog2e = 1.4426950408889634f;
  float s = 0.f;
  if (fabsf(m) < 65536.f) {
    const float c = m * kLog2e;
#pragma unroll
    for (int j = 0; j < J; ++j) ex[j] = ex2(fmaf(v[j], kLog2e, -c));
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) ex[j] = ex2((v[j] - m) * kLog2e);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) s += ex[j];
  return group_sum<W>(s);
}

// Keys in descending order (odd-even merge sort; J a power of two up to 8).
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }
template <typename K>
__device__ __forceinline__ void order2(K& a, K& b) {
  const K hi = larger(a, b);
  b = smaller(a, b);
  a = hi;
}
template <typename K, int J>
__device__ __forceinline__ void sort_down(K (&s)[J]) {
  if constexpr (J == 2) {
    order2(s[0], s[1]);
  } else if constexpr (J == 4) {
    order2(s[0], s[1]); order2(s[2], s[3]); order2(s[0], s[2]); order2(s[1], s[3]); order2(s[1], s[2]);
  } else if constexpr (J == 8) {
    order2(s[0], s[1]); order2(s[2], s[3]); order2(s[4], s[5]); order2(s[6], s[7]);
    order2(s[0], s[2]); order2(s[1], s[3]); order2(s[4], s[6]); order2(s[5], s[7]);
    order2(s[1], s[2]); order2(s[5], s[6]);
    order2(s[0], s[4]); order2(s[1], s[5]); order2(s[2], s[6]); order2(s[3], s[7]);
    order2(s[2], s[4]); order2(s[3], s[5]);
    order2(s[1], s[2]); order2(s[3], s[4]); order2(s[5], s[6]);
  }
}

// The k-th largest key of the group, `none` where there are fewer: every lane
// orders its own once, then k times the largest head of the group is taken off
// (in step where two lanes have the same one).
template <int W, int J, int KMAX, typename K>
__device__ __forceinline__ K kth_largest(const K (&key)[J], int k, K none) {
  constexpr int S = J < KMAX ? J : KMAX;
  K s[J];
#pragma unroll
  for (int j = 0; j < J; ++j) s[j] = key[j];
  sort_down<K, J>(s);
  K th = none;
#pragma unroll
  for (int i = 0; i < KMAX; ++i) {
    if (i < k) {
      th = s[0];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) th = larger(th, __shfl_xor_sync(0xffffffffu, th, o));
      const bool pop = s[0] == th;
#pragma unroll
      for (int j = 0; j + 1 < S; ++j) s[j] = pop ? s[j + 1] : s[j];
      s[S - 1] = pop ? none : s[S - 1];
    }
  }
  return th;
}

// The choices of a token by definition: k times the largest that is left, the
// first of equals.  Adds 1 to cn of the chosen ones.
template <int W, int J>
__device__ __forceinline__ void choose_ordered(const float (&v)[J], int e0, int k, float (&cn)[J]) {
  uint32_t taken = 0;
  for (int i = 0; i < k; ++i) {
    float best = -INFINITY;
    int at = 1 << 20;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (!(taken >> j & 1) && v[j] > best) { best = v[j]; at = e0 + j; }
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (ov > best || (ov == best && oa < at)) { best = ov; at = oa; }
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (at == e0 + j) { taken |= 1u << j; cn[j] += 1.f; }
  }
}

// The same by the k-th largest: what reaches it is chosen.
//
// fp32: where at most k values reach it they are the choices.  Ties at it, or
// above it (heads taken off in step, until none may be left), leave more than
// k, and the warp then chooses by definition.
//
// bf16 logits tie often, but fit the upper half of a 32-bit key whose lower
// half holds the expert's place: no two keys are equal, and their order is the
// one that ties ask for.  (The two zeros are made one first.)
template <typename XT, int W, int J, int KMAX>
__device__ __forceinline__ void choose(const float (&v)[J], int e0, int k, float (&cn)[J]) {
  if constexpr (sizeof(XT) == 2) {
    constexpr uint32_t kLowest = 0x007FFFFFu;  // the largest key of -inf
    uint32_t key[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t bits = __float_as_uint(v[j] + 0.f);
      const uint32_t sign = static_cast<uint32_t>(static_cast<int>(bits) >> 31);
      key[j] = __byte_perm(bits ^ (sign | 0x80000000u), 0xFFFFu - (e0 + j), 0x3254);
    }
    const uint32_t th = kth_largest<W, J, KMAX, uint32_t>(key, k, 0u);
#pragma unroll
    for (int j = 0; j < J; ++j) cn[j] += key[j] >= th && key[j] > kLowest ? 1.f : 0.f;
  } else {
    const float th = kth_largest<W, J, KMAX, float>(v, k, -INFINITY);
    float hit[J], mine = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      hit[j] = v[j] >= th && v[j] > -INFINITY ? 1.f : 0.f;
      mine += hit[j];
    }
    const float all = group_sum<W>(mine);
    if (__any_sync(0xffffffffu, all > static_cast<float>(k))) {
      choose_ordered<W, J>(v, e0, k, cn);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) cn[j] += hit[j];
    }
  }
}

// u = log(sigmoid(l)) and sg = sigmoid(-l)
__device__ __forceinline__ void log_sigmoid(float l, float& u, float& sg) {
  const float t = __expf(-fabsf(l));
  const float r = __fdividef(1.f, 1.f + t);
  u = fminf(l, 0.f) - __logf(1.f + t);
  sg = l >= 0.f ? t * r : r;
  if (!(l == l)) u = sg = l;  // NaN
}

template <typename XT, int W, int J, int KMAX, bool SIG>
__global__ void __launch_bounds__(THREADS, 4) balance_tile_kernel(const BalanceArgs a, int vec) {
  constexpr int ROWS = THREADS / W;
  __shared__ float s_p[ROWS][W * J];
  __shared__ int s_c[ROWS][W * J];
  __shared__ float s_z[ROWS];
  __shared__ int s_n[ROWS];
  const int row = threadIdx.x / W, l = threadIdx.x % W, e0 = l * J;
  const int E = a.E;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile, t1 = min(a.T, t0 + a.tile);
  float* slots = static_cast<float*>(a.workspace);
  pdl_wait();
  pdl_trigger();
  int64_t b = seq_of(a, t0), pos = t0;
  for (; b < a.B && pos < t1; ++b) {
    const int64_t s = max(seq_begin(a, b), pos), e = min(seq_begin(a, b + 1), t1);
    if (s >= t1) break;
    if (e <= s) continue;
    pos = e;
    float ps[J], cn[J], zs = 0.f;  // (counts in fp32: a tile holds far fewer than 2^24 tokens)
    int n = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) ps[j] = cn[j] = 0.f;
    // a token's logits are loaded while the one before is worked on
    const XT* src = static_cast<const XT*>(a.logits) + (s + row) * E;
    const uint8_t* mask = a.mask != nullptr ? a.mask + s + row : nullptr;
    const int left = static_cast<int>(e - s) - row;  // (at most a tile)
    auto load = [&](int i, float (&v)[J]) {  // the token i after this row's first
      if (i < left && (mask == nullptr || mask[i] != 0)) {
        load_logits<XT, J>(src, e0, E, vec, v);
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = -INFINITY;
      }
    };
    float v[J], nv[J];
    load(0, nv);
    for (int i = 0; i < static_cast<int>(e - s); i += ROWS) {  // (every lane of a warp runs the same steps)
#pragma unroll
      for (int j = 0; j < J; ++j) v[j] = nv[j];
      src += ROWS * E;
      load(i + ROWS, nv);
      float m = v[0];
#pragma unroll
      for (int j = 1; j < J; ++j) m = max_nan(m, v[j]);
      m = group_max<W>(m);
      const bool live = !(m == -INFINITY);  // no expert left (or none read): not a token that counts
      choose<XT, W, J, KMAX>(v, e0, a.k, cn);
      float ex[J];
      const float base = live ? m : 0.f;
      float sum = exp_sum<W, J>(v, base, ex);
      const float lse = base + logf(sum);
      if (SIG) {
        float u[J], sg;
#pragma unroll
        for (int j = 0; j < J; ++j) log_sigmoid(v[j], u[j], sg);
        float um, us;
        log_sigmoid(base, um, us);
        sum = exp_sum<W, J>(u, um, ex);
      }
      if (live) {
        const float r = __fdividef(1.f, sum);
#pragma unroll
        for (int j = 0; j < J; ++j) ps[j] = fmaf(ex[j], r, ps[j]);
        zs = fmaf(lse, lse, zs);
        n += 1;
      }
    }
    __syncthreads();  // (the last segment's sums have been read)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      s_p[row][e0 + j] = ps[j];
      s_c[row][e0 + j] = static_cast<int>(cn[j]);
    }
    if (l == 0) { s_z[row] = zs; s_n[row] = n; }
    __syncthreads();
    const int64_t slot = s == t0 ? 2 * static_cast<int64_t>(blockIdx.x) : e == t1 ? 2 * static_cast<int64_t>(blockIdx.x) + 1 : 2 * a.tiles + b;
    float* out = slots + slot * slot_words(E);
    for (int i = threadIdx.x; i <= E; i += THREADS) {
      if (i < E) {
        float p = 0.f;
        int c = 0;
#pragma unroll 8
        for (int r = 0; r < ROWS; ++r) { p += s_p[r][i]; c += s_c[r][i]; }
        out[i] = p;
        reinterpret_cast<int*>(out)[E + i] = c;
      } else {
        float z = 0.f;
        int nn = 0;
        for (int r = 0; r < ROWS; ++r) { z += s_z[r]; nn += s_n[r]; }
        out[2 * E] = z;
        reinterpret_cast<int*>(out)[2 * E + 1] = nn;
      }
    }
  }
}

// Adds the slots of one sequence in a fixed order and writes its results:
// thread (part, e) takes every parts-th slot's entry of expert e, thread t
// every FINAL-th slot's scalars from t on.
constexpr int FINAL = 512;

__global__ void __launch_bounds__(FINAL) balance_final_kernel(const BalanceArgs a) {
  __shared__ double s_p[FINAL];
  __shared__ int s_c[FINAL];
  __shared__ double s_dot[FINAL / 32], s_z[FINAL / 32];
  __shared__ int s_n[FINAL / 32];
  const int E = a.E;
  const int64_t b = blockIdx.x;
  const int64_t s = seq_begin(a, b), e = seq_begin(a, b + 1);  // (the caller's: not the kernel's before)
  pdl_wait();
  pdl_trigger();
  const float* slots = static_cast<const float*>(a.workspace);
  const int64_t c0 = s / a.tile, c1 = e > s ? (e - 1) / a.tile + 1 : c0;
  auto slot_of = [&](int64_t c) {
    const int64_t u0 = c * a.tile, u1 = min(a.T, u0 + a.tile);
    const int64_t at = max(s, u0) == u0 ? 2 * c : min(e, u1) == u1 ? 2 * c + 1 : 2 * a.tiles + b;
    return slots + at * slot_words(E);
  };
  int pe = 1;
  while (pe < E) pe <<= 1;
  const int parts = FINAL / pe, part = threadIdx.x / pe, ei = threadIdx.x % pe;
  double p = 0.0, z = 0.0;
  int cnt = 0, n = 0;
  if (ei < E) {
    int64_t c = c0 + part;
    for (; c + 3 * parts < c1; c += 4 * parts) {
      float v[4];
      int k[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* q = slot_of(c + i * parts);
        v[i] = q[ei];
        k[i] = reinterpret_cast<const int*>(q)[E + ei];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) { p += static_cast<double>(v[i]); cnt += k[i]; }
    }
    for (; c < c1; c += parts) {
      const float* q = slot_of(c);
      p += static_cast<double>(q[ei]);
      cnt += reinterpret_cast<const int*>(q)[E + ei];
    }
  }
  for (int64_t c = c0 + threadIdx.x; c < c1; c += FINAL) {
    const float* q = slot_of(c);
    z += static_cast<double>(q[2 * E]);
    n += reinterpret_cast<const int*>(q)[2 * E + 1];
  }
  s_p[threadIdx.x] = p;
  s_c[threadIdx.x] = cnt;
  __syncthreads();
  double dot = 0.0;
  if (threadIdx.x < E) {
    for (int i = 1; i < parts; ++i) { p += s_p[i * pe + ei]; cnt += s_c[i * pe + ei]; }
    a.counts[b * E + ei] = cnt;
    dot = p * static_cast<double>(cnt);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    dot += __shfl_xor_sync(0xffffffffu, dot, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if ((threadIdx.x & 31) == 0) {
    s_dot[threadIdx.x >> 5] = dot;
    s_z[threadIdx.x >> 5] = z;
    s_n[threadIdx.x >> 5] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < FINAL / 32; ++i) { dot += s_dot[i]; z += s_z[i]; n += s_n[i]; }
    const double dn = static_cast<double>(n);
    a.aux[b] = n > 0 ? static_cast<float>(static_cast<double>(E) * dot / (static_cast<double>(a.k) * dn * dn)) : 0.f;
    a.z[b] = n > 0 ? static_cast<float>(z / dn) : 0.f;
    a.tokens[b] = n;
  }
}

template <typename XT, int W, int J, bool SIG>
__global__ void __launch_bounds__(THREADS) balance_backward_kernel(const BalanceArgs a, int vec, int vec_out,
                                                                   int per_group) {
  constexpr int ROWS = THREADS / W;
  const int row = threadIdx.x / W, l = threadIdx.x % W, e0 = l * J;
  const int E = a.E;
  pdl_wait();
  pdl_trigger();
  const int T = static_cast<int>(a.T);  // below 2^31
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * ROWS + row) * per_group;
  const XT* src = static_cast<const XT*>(a.logits) + first * E;
  float* dst = a.dlogits + first * E + e0;
  const uint8_t* mask = a.mask != nullptr ? a.mask + first : nullptr;
  int t = first < T ? static_cast<int>(first) : T;  // (past T nothing is read or written)
  int64_t b = -1;
  int end = t;           // where the present coefficients end
  bool counts = false;   // the present token's sequence has tokens that count
  float g[J], dz2 = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) g[j] = 0.f;
  for (int i = 0; i < per_group; ++i, ++t, src += E, dst += E) {  // (every lane of a warp runs the same steps)
    if (t >= end && t < T) {  // the coefficients of t's sequence
      if (b < 0) b = seq_of(a, t);
      while (b + 1 < a.B && seq_begin(a, b + 1) <= t) ++b;
      const int lo = static_cast<int>(seq_begin(a, b)), hi = static_cast<int>(seq_begin(a, b + 1));
      const bool inside = t >= lo && t < hi;
      end = inside ? hi : t < lo ? lo : T;
      const float n = inside ? static_cast<float>(a.tokens_in[b]) : 0.f;
      counts = n > 0.f;
      const float r = counts ? 1.f / n : 0.f;
      const float ca = a.daux != nullptr && counts ? a.daux[b] * static_cast<float>(E) / static_cast<float>(a.k) * r * r : 0.f;
      const float mean = static_cast<float>(a.k) * n / static_cast<float>(E);
      dz2 = a.dz != nullptr && counts ? a.dz[b] * 2.f * r : 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
        g[j] = counts && e0 + j < E ? ca * (static_cast<float>(a.counts_in[b * E + e0 + j]) - mean) : 0.f;
    }
    const bool in = t < T && counts && (mask == nullptr || mask[i] != 0);
    float v[J];
    if (in) {
      load_logits<XT, J>(src, e0, E, vec, v);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) v[j] = -INFINITY;
    }
    float m = v[0];
#pragma unroll
    for (int j = 1; j < J; ++j) m = max_nan(m, v[j]);
    m = group_max<W>(m);
    const bool live = in && !(m == -INFINITY);
    const float base = live ? m : 0.f;
    float ex[J], d[J];
    const float sum = exp_sum<W, J>(v, base, ex);
    const float zc = dz2 * (base + logf(sum)) * __fdividef(1.f, sum);
    if (SIG) {
      float u[J], sg[J], pu[J], um, us;
#pragma unroll
      for (int j = 0; j < J; ++j) log_sigmoid(v[j], u[j], sg[j]);
      log_sigmoid(base, um, us);
      const float r = __fdividef(1.f, exp_sum<W, J>(u, um, pu));
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) { pu[j] *= r; dot = fmaf(pu[j], g[j], dot); }
      dot = group_sum<W>(dot);
#pragma unroll
      for (int j = 0; j < J; ++j) d[j] = fmaf(ex[j], zc, pu[j] * (g[j] - dot) * sg[j]);
    } else {
      const float r = __fdividef(1.f, sum);
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) dot = fmaf(ex[j], g[j], dot);
      dot = group_sum<W>(dot) * r;
#pragma unroll
      for (int j = 0; j < J; ++j) d[j] = ex[j] * fmaf(r, g[j] - dot, zc);
    }
    if (t < T) {
      if (J >= 4 && vec_out && e0 + J <= E) {
#pragma unroll
        for (int j = 0; j < J; j += 4)
          *reinterpret_cast<float4*>(dst + j) = live ? make_float4(d[j], d[(j + 1) % J], d[(j + 2) % J], d[(j + 3) % J])
                                                   : make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (e0 + j < E) dst[j] = live ? d[j] : 0.f;
      }
    }
  }
}

template <typename XT, int W, int J, bool SIG>
cudaError_t launch_w(const BalanceArgs& a, bool backward, cudaStream_t s) {
  const int vec = ((reinterpret_cast<uintptr_t>(a.logits) | (a.E * sizeof(XT))) & 15) == 0;
  if (!backward) {
    const cudaError_t e = a.tiles == 0 ? cudaSuccess
                          : a.k <= 4 ? launch_pdl(balance_tile_kernel<XT, W, J, 4, SIG>, dim3(static_cast<unsigned>(a.tiles)),
                                                  dim3(THREADS), 0, s, a, vec)
                                     : launch_pdl(balance_tile_kernel<XT, W, J, 8, SIG>, dim3(static_cast<unsigned>(a.tiles)),
                                                  dim3(THREADS), 0, s, a, vec);
    if (e != cudaSuccess) return e;
    return launch_pdl(balance_final_kernel, dim3(static_cast<unsigned>(a.B)), dim3(FINAL), 0, s, a);
  }
  const int vec_out = ((reinterpret_cast<uintptr_t>(a.dlogits) | (a.E * sizeof(float))) & 15) == 0;
  constexpr int ROWS = THREADS / W;
  // consecutive tokens of a group of lanes share their sequence's coefficients
  const int per = static_cast<int>(std::min<int64_t>(8, std::max<int64_t>(1, a.T / (int64_t{ROWS} * 148 * 8))));
  const int64_t blocks = (a.T + static_cast<int64_t>(ROWS) * per - 1) / (static_cast<int64_t>(ROWS) * per);
  return launch_pdl(balance_backward_kernel<XT, W, J, SIG>, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, s, a,
                    vec, vec_out, per);
}

template <typename XT, bool SIG>
cudaError_t launch_e(const BalanceArgs& a, bool backward, cudaStream_t s) {
  if (a.E <= 8) return launch_w<XT, 8, 1, SIG>(a, backward, s);
  if (a.E <= 16) return launch_w<XT, 8, 2, SIG>(a, backward, s);
  if (a.E <= 32) return launch_w<XT, 8, 4, SIG>(a, backward, s);
  if (a.E <= 64) return launch_w<XT, 8, 8, SIG>(a, backward, s);
  if (a.E <= 128) return launch_w<XT, 16, 8, SIG>(a, backward, s);
  return launch_w<XT, 32, 8, SIG>(a, backward, s);
}

cudaError_t launch_any(const BalanceArgs& a, bool backward, cudaStream_t s) {
  if (a.is_bf16)
    return a.sigmoid ? launch_e<__nv_bfloat16, true>(a, backward, s) : launch_e<__nv_bfloat16, false>(a, backward, s);
  return a.sigmoid ? launch_e<float, true>(a, backward, s) : launch_e<float, false>(a, backward, s);
}

}  // namespace

int balance_tile(int64_t T) {
  const int64_t t = (T + 148 * 4 - 1) / (148 * 4);
  return static_cast<int>(std::max<int64_t>(32, (t + 31) / 32 * 32));
}

size_t balance_workspace_bytes(int64_t T, int E, int64_t B) {
  const int64_t tile = balance_tile(T), tiles = (T + tile - 1) / tile;
  return sizeof(float) * static_cast<size_t>(2 * tiles + B) * static_cast<size_t>(slot_words(E));
}

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) { return launch_any(a, false, s); }
cudaError_t launch_balance_backward(const BalanceArgs& a, cudaStream_t s) { return launch_any(a, true, s); }

}  // namespace moe
