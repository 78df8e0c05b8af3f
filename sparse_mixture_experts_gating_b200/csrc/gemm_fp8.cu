// Grouped product of two e4m3 operands with block scales on the 5th-generation
// tensor cores (tcgen05 + TMEM), fed by TMA:
//
//   y[r][n] = sum_kb sa[r][kb] sb[n or n / 128][kb] sum_{k in block kb} A[r][k] B_g[n][k]
//
// for the rows r of every group g (offsets on the device; one group without
// them).  The scales are arbitrary fp32 numbers, so the tensor core sums one
// k-block of 128 (one 128-byte swizzled row of shared memory, four MMAs of
// K = 32) into its own TMEM accumulator, and the summing warps read it back,
// multiply by sa * sb and add it to fp32 registers while the next k-block's
// MMAs fill the other accumulator.  Tiles are 128 rows x 256 columns.
//
// What bounds it, by form:
//
// Many rows, scales of 128 x 128 weights: alone, a k-block's MMAs take 514 cycles,
// its 32768 additions 256 (the fp32 rate of an SM) and its read-back 144.  Together
// a k-block takes 930: the MMAs 720, the summing warps 730 and a wait of 200, for
// the read-back shares TMEM with the accumulation (counters: tensor pipe 54 %
// active, shared memory's banks 20 % reads and 20 % writes).  8192 x 14336 x 4096: 456 us in bursts (2.1
// PFLOP/s), 507-542 us back to back, where the board's power limit sets the
// clock (cuBLAS with one scale per tensor: 331 and 385 us).  Eight summing warps
// of 128 columns with 232 registers each were the fastest of the forms tried;
// sixteen of 64 columns, MMAs of half the width with four accumulators, and
// sums kept in register pairs took 1.1 to 1.4 times as long.
// A scale for every column (SB1): each summing warp reads 128 column scales and
// multiplies by them as well, 1.5 times as long (4736 x 4096 x 4096: 114 and 76.5 us).
// Few k-blocks a tile: the epilogue, about 5 k-blocks long, is not hidden (128
// ragged groups, 40961 x 768 x 2048: 95 us in bursts, eight tiles of 16 k-blocks a
// CTA, of whose rows a sixth belong to no group).
// A few rows: a k-block still costs its whole loop, 0.42 us with weights in L2 and
// few CTAs, and HBM serves about 90 CTAs at that pace; the launch, the first loads
// and the cluster's meeting are 5 us (one token times 14336 x 4096: 15.3 us, 12.2 with
// the weights in L2).
//
// Warp roles (384 threads, one CTA per SM):
//   warp 0       TMA producer
//   warp 1       TMEM allocator; lane 0 issues tcgen05.mma
//   warp 3       column scales (SB1)
//   warps 4..11  summing and epilogue: warp w owns TMEM lanes 32 (w % 4) ..
//                (rows of the tile) and the columns of half (w - 4) / 4
//   (warps 0..3 are the warpgroup that gives its registers to the other two)
// Pipelines: a ring of shared-memory stages (full / empty) and two TMEM
// accumulators of 256 columns (tfull / tempty), one k-block each.  Every wait
// is bounded; one that runs out records MOE_ERR_TIMEOUT, raises the CTA's
// abort flag, and the CTA drains its copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "internal.h"

namespace moe {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;                 // e4m3 elements per 128-byte shared-memory row
constexpr int MMA_N = 256;
constexpr int B_HALF = 128 * BK;        // 16 KB per 128 rows of B
constexpr int MAX_STAGES = 6;
constexpr int NUM_THREADS = 384;
// 384 threads start with 168 registers each; the first warpgroup gives most of
// its share to the two that hold the fp32 sums: 40 + 2 x 232 = 3 x 168.
constexpr int REGS_START = 168, REGS_FEED = 40, REGS_SUM = 232;
static_assert(REGS_FEED + 2 * REGS_SUM <= 3 * REGS_START, "the registers of the launch");
constexpr int EPI_WARPS = 8;
// Column scales (SB1): a ring of SB_ROWS k-blocks, copied SB_KB at a time, in rows of
// SB_LD floats, a bank apart by 8 so that 8 columns x 4 k-blocks take all 32.
constexpr int SB_ROWS = 12, SB_KB = 4, SB_LD = MMA_N + 8;
constexpr uint32_t TMEM_COLS = 2 * MMA_N;
constexpr int ROW_STAGE = 64;           // bytes per staged output row of a warp's own stores
constexpr int CL_ROWS = 8;              // rows of a product whose CTAs may sum in clusters
constexpr int CL_LD = MMA_N + 4;        // floats between the rows of a sum handed to the cluster's first CTA
constexpr int MAX_CLUSTER = 8;
constexpr int OUT_HALF = 2 * 16384;     // two boxes of 128 rows x 128 bytes of a warpgroup's TMA stores

// AR: rows of A a stage holds.  No group has more rows than max_group_rows, so
// a small batch stages 32 or 64 and keeps more weight bytes in flight; the
// M = 128 MMA then reads the bytes that follow, which only feed accumulator
// rows that are never stored.
//
// OUT_BYTES: where the summing warps lay out what they store.  With whole
// tiles (AR 128) a warpgroup lays out 128 rows x 256 bytes and stores them by
// TMA under the next tile's products: stored by the threads themselves, every
// CTA's tile at the same time, a tile's 64 KB took 6200 cycles of 32000.  That
// leaves room for three stages instead of four.
template <int AR>
struct Geo {
  static constexpr int A_ST = AR * BK;
  static constexpr int STAGE_BYTES = A_ST + 2 * B_HALF;
  static constexpr int OUT_BYTES = AR == BM ? 2 * OUT_HALF : EPI_WARPS * 32 * ROW_STAGE;
  static constexpr int ROOM = 226 * 1024 - 6 * 1024 - OUT_BYTES;
  static constexpr int STAGES = (ROOM / STAGE_BYTES) < MAX_STAGES ? (ROOM / STAGE_BYTES) : MAX_STAGES;
};

struct Ctl {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_slot;
  volatile int abort;
  int mprefix[kFp8MaxGroups + 1];
  int offsets[kFp8MaxGroups + 1];
  float hmax[2][BM];
};

// Byte offset of 16-byte piece v of staged row r: the pieces are permuted so that
// eight rows written at one v, and two rows read at four, take all 32 banks.
__device__ __forceinline__ int stage_at(int r, int v) { return r * ROW_STAGE + ((v ^ (r >> 1 & 3)) << 4); }

constexpr size_t CTL_BYTES = (sizeof(Ctl) + 15) / 16 * 16;

template <int AR, bool SB1>
constexpr size_t smem_bytes() {
  return Geo<AR>::STAGES * Geo<AR>::STAGE_BYTES + Geo<AR>::OUT_BYTES + CTL_BYTES +
         (SB1 ? sizeof(float) * SB_ROWS * SB_LD : 0) + 1024;
}

// kind::f8f6f4: e4m3 A and B (format fields 0, both K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Group tables from the caller's offsets, clamped into [0, rows] and made
// ascending by a running maximum (a bad table can give wrong rows, never an
// access outside the buffers): offsets and the running count of 128-row tiles.
// One warp; lane l takes groups 8 l .. 8 l + 7.
__device__ __forceinline__ void load_groups(Ctl* c, const Fp8Params& p, int lane) {
  static_assert(kFp8MaxGroups == 256, "eight groups per lane");
  const int rows = static_cast<int>(p.a_rows);
  if (p.offsets == nullptr) {
    if (lane == 0) {
      c->offsets[0] = 0;
      c->offsets[1] = rows;
      c->mprefix[0] = 0;
      c->mprefix[1] = (rows + BM - 1) / BM;
    }
    return;
  }
  const int first = min(max(p.offsets[0], 0), rows);
  int end[8];  // offsets[g + 1]
  int run = first;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int g = lane * 8 + i;
    const int o = g < p.G ? min(max(p.offsets[g + 1], 0), rows) : 0;
    run = max(run, o);
    end[i] = run;
  }
  int before = run;  // running maximum over the lanes below
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before = max(before, v);
  }
  before = __shfl_up_sync(0xffffffffu, before, 1);
  if (lane == 0) before = first;
  int tiles = 0, prev = before;
  int cum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    end[i] = max(end[i], before);
    tiles += (end[i] - prev + BM - 1) / BM;
    prev = end[i];
    cum[i] = tiles;
  }
  int sum = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  const int base = sum - tiles;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int g = lane * 8 + i;
    if (g < p.G) {
      c->offsets[g + 1] = end[i];
      c->mprefix[g + 1] = base + cum[i];
    }
  }
  if (lane == 0) {
    c->offsets[0] = first;
    c->mprefix[0] = 0;
  }
}

// Unit u of the work: tile u / ksplit (group-major, then column tile, then row
// tile, so that tiles sharing B run together), K range u % ksplit.
struct Item {
  int g, mt, nt, ks, kb0, kb1;
};
__device__ __forceinline__ bool item_at(const Ctl* c, const Fp8Params& p, int64_t u, Item& w) {
  if (u >= static_cast<int64_t>(c->mprefix[p.G]) * p.n_tiles * p.ksplit) return false;
  const int t = static_cast<int>(u / p.ksplit);
  w.ks = static_cast<int>(u - static_cast<int64_t>(t) * p.ksplit);
  int lo = 0, hi = p.G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c->mprefix[mid] * p.n_tiles <= t) lo = mid; else hi = mid;
  }
  w.g = lo;
  const int local = t - c->mprefix[lo] * p.n_tiles;
  const int mtiles = c->mprefix[lo + 1] - c->mprefix[lo];
  w.nt = local / mtiles;
  w.mt = local - w.nt * mtiles;
  w.kb0 = w.ks * p.kb_per;
  w.kb1 = min(p.num_kb, w.kb0 + p.kb_per);
  return true;
}

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// One fp32 number, copied without waiting.
__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrive on `bar` (within its count) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for the warp's TMEM loads; t passes through, so that no use of it moves up.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&t)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(t[0]), "+r"(t[1]), "+r"(t[2]), "+r"(t[3]), "+r"(t[4]), "+r"(t[5]), "+r"(t[6]), "+r"(t[7]),
                 "+r"(t[8]), "+r"(t[9]), "+r"(t[10]), "+r"(t[11]), "+r"(t[12]), "+r"(t[13]), "+r"(t[14]), "+r"(t[15]),
                 "+r"(t[16]), "+r"(t[17]), "+r"(t[18]), "+r"(t[19]), "+r"(t[20]), "+r"(t[21]), "+r"(t[22]), "+r"(t[23]),
                 "+r"(t[24]), "+r"(t[25]), "+r"(t[26]), "+r"(t[27]), "+r"(t[28]), "+r"(t[29]), "+r"(t[30]), "+r"(t[31])
               :
               : "memory");
}

// d = a * b + d on two fp32 numbers at once.
__device__ __forceinline__ void fma2(float& d0, float& d1, uint32_t a0, uint32_t a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}\n"
      : "+f"(d0), "+f"(d1)
      : "r"(a0), "r"(a1), "f"(b0), "f"(b1));
}

// d = a * (b * s) + d on two fp32 numbers at once.
__device__ __forceinline__ void mul_fma2(float& d0, float& d1, uint32_t a0, uint32_t a1, float b0, float b1, float s) {
  asm("{\n\t.reg .b64 x, y, z, q;\n\t"
      "mov.b64 q, {%6, %6};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 y, y, q;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}\n"
      : "+f"(d0), "+f"(d1)
      : "r"(a0), "r"(a1), "f"(b0), "f"(b1), "f"(s));
}

// Every thread of the cluster's CTAs meets here (what was written before is seen after).
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of p (this CTA's shared memory) in the cluster's first CTA, and a store to such an address.
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void st_cluster4(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// acc[i] += t[i] * (a scale): one scale for all 32 columns, or (SB1) s times one for each in `b`.
template <bool SB1>
__device__ __forceinline__ void add32(float* acc, const uint32_t (&t)[32], float s, const float* b) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    if (SB1) {
      const float4 v = *reinterpret_cast<const float4*>(b + i);
      mul_fma2(acc[i], acc[i + 1], t[i], t[i + 1], v.x, v.y, s);
      mul_fma2(acc[i + 2], acc[i + 3], t[i + 2], t[i + 3], v.z, v.w, s);
    } else {
      fma2(acc[i], acc[i + 1], t[i], t[i + 1], s, s);
      fma2(acc[i + 2], acc[i + 3], t[i + 2], t[i + 3], s, s);
    }
  }
}

// silu(a) * b from the special function unit's exponential and reciprocal (each
// good to two units, and the exponential's argument, rounded, moves it by up to
// |a| units more: codes have 4 bits of the 24; 0 once e^-a overflows, the limit of
// silu, whatever a b is).
__device__ __forceinline__ float silu_mul(float a, float b) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return a * r * b;
}

// 16 bytes of an output row: eight bf16, eight fp16 scaled by g, or four fp32 times g.
template <int EPI>
__device__ __forceinline__ uint4 out_piece(const float* s, float g) {
  if constexpr (EPI == FP8_BF16) {
    return make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
  } else if constexpr (EPI == FP8_GATE_H16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(s[2 * i] * g, s[2 * i + 1] * g);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(__float_as_uint(s[0] * g), __float_as_uint(s[1] * g), __float_as_uint(s[2] * g),
                      __float_as_uint(s[3] * g));
  }
}

template <int BYTES>
struct OutWord { using type = uint16_t; };
template <>
struct OutWord<4> { using type = uint32_t; };

// CLUSTER: one item a CTA, its K ranges summed within a cluster (p.cluster CTAs).
template <int EPI, int AR, bool SB1, bool CLUSTER>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                    const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmOut, const Fp8Params p) {
  constexpr bool PAIR = EPI == FP8_SWIGLU || EPI == FP8_PAIR_F32;  // 128 columns of W1 and the same of W3
  constexpr bool F32 = EPI == FP8_F32 || EPI == FP8_PAIR_F32;
  constexpr bool ACT = EPI == FP8_SWIGLU || EPI == FP8_RELU;
  static_assert(!CLUSTER || (AR < BM && (EPI == FP8_BF16 || EPI == FP8_F32)), "products of few rows");
  constexpr uint32_t IDESC = idesc_e4m3_f32(BM, MMA_N);
  using G = Geo<AR>;
  constexpr int STAGES = G::STAGES, STAGE_BYTES = G::STAGE_BYTES, A_ST = G::A_ST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* out_stage = stages + STAGES * STAGE_BYTES;
  Ctl* ctl = reinterpret_cast<Ctl*>(out_stage + G::OUT_BYTES);
  float* sb_ring = reinterpret_cast<float*>(out_stage + G::OUT_BYTES + CTL_BYTES);  // SB1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&ctl->full[s], SB1 ? 33 : 1); mbar_init(&ctl->empty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&ctl->tfull[a], 1); mbar_init(&ctl->tempty[a], EPI_WARPS); }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB0);
    if (PAIR) tma_prefetch_desc(&tmB1);
  }
  if (warp == 1) tmem_alloc(&ctl->tmem_slot, TMEM_COLS);
  pdl_wait();  // the operands and the group table come from the kernels before
  pdl_trigger();
  if (warp == 2) load_groups(ctl, p, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_slot;
  Item w;

  if (warp < 4) {
    reg_dec<REGS_FEED>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (int64_t u = blockIdx.x; ok && item_at(ctl, p, u, w); u += gridDim.x) {
        const int row0 = ctl->offsets[w.g] + w.mt * BM;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait_or_abort(&ctl->empty[stage], phase ^ 1u, &ctl->abort, p.err, p.limit_ns)) { ok = false; break; }
          uint8_t* sa = stages + stage * STAGE_BYTES;
          mbar_arrive_expect_tx(&ctl->full[stage], A_ST + 2 * B_HALF);
          tma_load_2d(sa, &tmA, &ctl->full[stage], kb * BK, row0);
          if (PAIR) {
            tma_load_3d(sa + A_ST, &tmB0, &ctl->full[stage], kb * BK, w.nt * 128, w.g);
            tma_load_3d(sa + A_ST + B_HALF, &tmB1, &ctl->full[stage], kb * BK, w.nt * 128, w.g);
          } else {
            tma_load_3d(sa + A_ST, &tmB0, &ctl->full[stage], kb * BK, w.nt * 256, w.g);  // 256-row box
          }
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // Drain: every issued copy must have landed before the CTA may exit.
      for (int s = 0; s < STAGES; ++s)
        if ((issued >> s) & 1u) mbar_wait(&ctl->full[s], (issued_phase >> s) & 1u, p.limit_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t u = blockIdx.x; ok && item_at(ctl, p, u, w); u += gridDim.x) {
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait_or_abort(&ctl->tempty[acc], acc_phase ^ 1u, &ctl->abort, p.err, p.limit_ns) ||
              !mbar_wait_or_abort(&ctl->full[stage], phase, &ctl->abort, p.err, p.limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(stages + stage * STAGE_BYTES);
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * MMA_N);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            umma_f8(d_tmem, sdesc_k_sw128(sa + k * 32), sdesc_k_sw128(sa + A_ST + k * 32), IDESC, k != 0 ? 1u : 0u);
          umma_commit(&ctl->empty[stage]);
          umma_commit(&ctl->tfull[acc]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
      // Drain: all MMAs of this CTA complete before TMEM is freed.
      umma_commit(&ctl->drain);
      mbar_wait(&ctl->drain, 0, p.limit_ns);
    }
  } else if (SB1 && warp == 3) {
    // ------------------------------------------------------------ column scales
    // Neighbouring columns' scales lie a row of B's scales apart.  A lane copies
    // one k-block of a column, four lanes the chunk's, so that a request takes 8
    // cache lines and a sector's neighbours are taken with it (k-block by k-block
    // for 32 columns, 32 lines each, 4736 x 4096 x 4096 took 140 us).
    //
    // They need no barriers of their own (which cost every summing warp a wait and
    // an arrival: 128 us against 115): a k-block's stage is full once its scales have landed
    // too, so its MMAs' commit stands for both.  And k-block n is copied for after
    // its stage came free, which is after the MMAs of k-block n - STAGES, which
    // waited for the accumulator that the summing warps left before k-block n -
    // STAGES - 1: their scales up to n - STAGES - 3 have been read.
    static_assert(SB_KB - 1 - SB_ROWS <= -STAGES - 3 && SB_ROWS % SB_KB == 0, "the last row that a copy takes over has been read");
    const int kl = lane & (SB_KB - 1), cl = lane >> 2;
    int stage = 0, row = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; ok && item_at(ctl, p, u, w); u += gridDim.x) {
      const int col = w.nt * 256 + cl;
      const float* sb = p.sb0 + w.g * p.sb_gs + static_cast<int64_t>(col) * p.num_kb + kl;
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait_or_abort(&ctl->empty[stage], phase ^ 1u, &ctl->abort, p.err, p.limit_ns));
        if (!ok) break;
        if (((kb - w.kb0) & (SB_KB - 1)) == 0 && kb + kl < w.kb1) {
          int to = row + kl;
          if (to >= SB_ROWS) to -= SB_ROWS;
          float* dst = sb_ring + to * SB_LD + cl;
#pragma unroll 8
          for (int i = 0; i < MMA_N; i += 8)
            if (col + i < p.N) cp_async4(dst + i, sb + static_cast<int64_t>(i) * p.num_kb + kb);
        }
        cp_async_arrive(&ctl->full[stage]);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        if (++row == SB_ROWS) row = 0;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  } else {
    // ------------------------------------------------------------ summing and epilogue
    reg_inc<REGS_SUM>();
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int r_in_tile = q * 32 + lane;
    uint8_t* stg = out_stage + (warp - 4) * (G::OUT_BYTES / EPI_WARPS);
    constexpr bool TMA_OUT = AR == BM && EPI != FP8_PAIR_F32;
    const bool storer = (threadIdx.x & 127) == 0;  // issues its warpgroup's TMA stores (ACT: the first one both's)
    // PAIR: columns [64 half, +64) of W1, then of W3; else columns [128 half, +128)
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t col0 = PAIR ? 64u * half : 128u * half, col2 = PAIR ? 128u + 64u * half : 128u * half + 64u;
    int acc_i = 0, sb_row = 0;
    bool met = false;  // CLUSTER
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; ok && item_at(ctl, p, u, w); u += gridDim.x) {
      const int m_local = w.mt * BM + r_in_tile;
      const int row = ctl->offsets[w.g] + m_local;
      const bool vrow = row < ctl->offsets[w.g + 1];
      const bool warp_live = __any_sync(0xffffffffu, vrow);
      // scales: this row's of A, and of B's 128-row block(s)
      const int bn_blocks = (p.N + 127) >> 7;
      const int nb = PAIR ? w.nt : min(2 * w.nt + half, bn_blocks - 1);
      const float* sa = p.sa + (vrow ? static_cast<int64_t>(row) : 0) * p.sa_ld;
      const float* sb0 = p.sb0 + w.g * p.sb_gs + (SB1 ? 0 : static_cast<int64_t>(nb) * p.num_kb);
      const float* sb1 = PAIR ? p.sb1 + w.g * p.sb_gs + static_cast<int64_t>(nb) * p.num_kb : nullptr;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      // The scales of a k-block are fetched two blocks ahead.
      auto scale_a = [&](int kb) { return vrow && kb < w.kb1 ? __ldg(sa + kb) : 0.f; };
      auto scale_b0 = [&](int kb) { return !SB1 && kb < w.kb1 ? __ldg(sb0 + kb) : 1.f; };
      auto scale_b1 = [&](int kb) { return PAIR && kb < w.kb1 ? __ldg(sb1 + kb) : 1.f; };
      float a0 = scale_a(w.kb0), a1 = scale_a(w.kb0 + 1), b0 = scale_b0(w.kb0), b1 = scale_b0(w.kb0 + 1);
      float c0 = scale_b1(w.kb0), c1 = scale_b1(w.kb0 + 1);
#pragma unroll 1
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        const float s0 = a0 * b0, s1 = PAIR ? a0 * c0 : s0;
        a0 = a1; b0 = b1; c0 = c1;
        a1 = scale_a(kb + 2);
        b1 = scale_b0(kb + 2);
        c1 = scale_b1(kb + 2);
        const float* sbs = sb_ring + sb_row * SB_LD + half * 128;
        ok = ok && __all_sync(0xffffffffu,
                              mbar_wait_or_abort(&ctl->tfull[acc_i], acc_phase, &ctl->abort, p.err, p.limit_ns));
        if (ok) {
          tc_fence_after();
          if (warp_live) {
            // each load of 32 columns is in flight while the 32 before are added
            const uint32_t tb = lane_base + static_cast<uint32_t>(acc_i * MMA_N);
            uint32_t t[32], v[32];
            tmem_ld32(tb + col0, t);
            tmem_ld_wait32(t);
            tmem_ld32(tb + col0 + 32, v);
            add32<SB1>(acc, t, s0, sbs);
            tmem_ld_wait32(v);
            tmem_ld32(tb + col2, t);
            add32<SB1>(acc + 32, v, s0, sbs + 32);
            tmem_ld_wait32(t);
            tmem_ld32(tb + col2 + 32, v);
            add32<SB1>(acc + 64, t, s1, sbs + 64);
            tmem_ld_wait32(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[acc_i]);
            add32<SB1>(acc + 96, v, s1, sbs + 96);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[acc_i]);
          }
        }
        if (SB1 && ++sb_row == SB_ROWS) sb_row = 0;
        if (++acc_i == 2) { acc_i = 0; acc_phase ^= 1u; }
        if (!ok) break;
      }
      // A cluster's CTAs hold the sums of their K ranges: the others' go to the
      // first one, where the stages lay, and it adds them in order.  (One item a CTA.)
      bool mine = true;
      if constexpr (CLUSTER) {
        cluster_meet();  // the first CTA's MMAs have read its stages
        float* part = reinterpret_cast<float*>(stages) + r_in_tile * CL_LD + half * 128;
        if (w.ks > 0 && vrow) {
          const uint32_t to = in_first_cta(part + (w.ks - 1) * CL_ROWS * CL_LD);
#pragma unroll
          for (int i = 0; i < 128; i += 4) st_cluster4(to + i * 4, acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        }
        cluster_meet();
        mine = w.ks == 0;
        if (mine && vrow) {
          for (int k = 1; k < p.cluster; ++k, part += CL_ROWS * CL_LD) {
#pragma unroll
            for (int i = 0; i < 128; i += 4) {
              const float4 v = *reinterpret_cast<const float4*>(part + i);
              acc[i] += v.x; acc[i + 1] += v.y; acc[i + 2] += v.z; acc[i + 3] += v.w;
            }
          }
        }
        met = true;
      }
      // Where warps meet at barriers, they leave an aborted CTA together.  (Also:
      // the last tile's hmax has been read, and its stores have read out_stage.)
      if (TMA_OUT && storer) bulk_wait_read();
      if (EPI == FP8_SWIGLU || (EPI == FP8_RELU && TMA_OUT)) ok = named_barrier_and(3, 256, ok);
      else if (TMA_OUT) ok = named_barrier_and(1 + half, 128, ok);
      // FP8_GATE_H16: this row's 128 columns by one power of two
      float h16_scale = 1.f;
      if (EPI == FP8_GATE_H16) {
        float m = 0.f;
        const int n0 = w.nt * 256 + half * 128;
        if (n0 + 128 <= p.N) {
#pragma unroll
          for (int i = 0; i < 128; ++i) m = fmaxf(m, fabsf(acc[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 128; ++i) m = fmaxf(m, n0 + i < p.N ? fabsf(acc[i]) : 0.f);
        }
        const float g = vrow ? p.row_gate[row] : 0.f;
        const int ex = static_cast<int>(__float_as_uint(fabsf(m * g)) >> 23);  // 2^(ex - 127) <= m g < 2^(ex - 126)
        const int inv = max(ex - 14, 1);
        h16_scale = g * __uint_as_float(static_cast<uint32_t>(254 - inv) << 23);
        if (vrow && n0 < p.N)
          p.out_scales[static_cast<int64_t>(row) * ((p.N + 127) >> 7) + (n0 >> 7)] = __uint_as_float(static_cast<uint32_t>(inv) << 23);
      }
      const bool by_tma = TMA_OUT && p.tma_out && ctl->offsets[w.g] + w.mt * BM + BM <= ctl->offsets[w.g + 1];
      if (ACT) {
        // activation, then codes with one scale for each 128 columns of a row
        constexpr int NV = PAIR ? 64 : 128;
        const int n0 = PAIR ? w.nt * 128 + half * 64 : w.nt * 256 + half * 128;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          acc[i] = PAIR ? silu_mul(acc[i], acc[(i + 64) & 127]) : max_nan(acc[i], 0.f);
          m = fmaxf(m, fabsf(acc[i]));
        }
        if (n0 + NV > p.N) {  // columns past N are not the row's
          m = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) m = fmaxf(m, n0 + i < p.N ? fabsf(acc[i]) : 0.f);
        }
        if (PAIR) {  // the row's other 64 columns are with the other half's thread
          ctl->hmax[half][r_in_tile] = m;
          named_barrier(3, 256);
          m = fmaxf(m, ctl->hmax[half ^ 1][r_in_tile]);
        }
        const Fp8Scale s = fp8_scale(m);
        if (ok && vrow && n0 < p.N && (!PAIR || half == 0)) p.out_scales[static_cast<int64_t>(row) * bn_blocks + (n0 >> 7)] = s.scale;
        if (ok && vrow && n0 < p.N) {
          uint8_t* dst = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(row) * p.ld_out + n0;
          // PAIR: one box of 128 columns for both halves, else one for each
          uint8_t* box = out_stage + (PAIR ? 0 : half * OUT_HALF) + r_in_tile * 128;
          const int first = PAIR ? half * 4 : 0;
#pragma unroll
          for (int i = 0; i < NV; i += 16) {
            const uint4 v = make_uint4(
                e4m3x4(acc[i] * s.inv, acc[i + 1] * s.inv, acc[i + 2] * s.inv, acc[i + 3] * s.inv),
                e4m3x4(acc[i + 4] * s.inv, acc[i + 5] * s.inv, acc[i + 6] * s.inv, acc[i + 7] * s.inv),
                e4m3x4(acc[i + 8] * s.inv, acc[i + 9] * s.inv, acc[i + 10] * s.inv, acc[i + 11] * s.inv),
                e4m3x4(acc[i + 12] * s.inv, acc[i + 13] * s.inv, acc[i + 14] * s.inv, acc[i + 15] * s.inv));
            if (by_tma) *reinterpret_cast<uint4*>(box + (((first + i / 16) ^ (r_in_tile & 7)) << 4)) = v;
            else if (n0 + i < p.N) *reinterpret_cast<uint4*>(dst + i) = v;  // N is a multiple of 16
          }
        }
        if (by_tma && ok) {
          fence_async_shared();
          named_barrier(3, 256);
          if (storer && (!PAIR || half == 0) && n0 < p.N) {
            tma_store_3d(&tmOut, out_stage + (PAIR ? 0 : half * OUT_HALF), n0, ctl->offsets[w.g] + w.mt * BM, 0);
            bulk_commit();
          }
        }
      } else if (by_tma && ok) {
        // a row's 128 bytes in each box, its 16-byte pieces permuted as the map's swizzle has them
        constexpr int ELT = EPI == FP8_BF16 || EPI == FP8_GATE_H16 ? 2 : 4, BOX = 128 / ELT;
        const float g = (F32 && p.row_gate != nullptr && vrow) ? p.row_gate[row] : 1.f;
        const int n0 = w.nt * 256 + half * 128;
        uint8_t* boxes = out_stage + half * OUT_HALF;
#pragma unroll
        for (int r = 0; r < 128 / BOX / 2; ++r) {  // two boxes at a time
          if (r > 0) {
            if (storer) bulk_wait_read();
            named_barrier(1 + half, 128);
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const float* s = acc + (r * 2 + b) * BOX + v * (16 / ELT);
              const uint4 q = out_piece<EPI>(s, EPI == FP8_GATE_H16 ? h16_scale : g);
              *reinterpret_cast<uint4*>(boxes + b * 16384 + r_in_tile * 128 + ((v ^ (r_in_tile & 7)) << 4)) = q;
            }
          }
          fence_async_shared();
          named_barrier(1 + half, 128);
          if (storer) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int col = n0 + (r * 2 + b) * BOX;
              if (col < p.N) tma_store_3d(&tmOut, boxes + b * 16384, col, ctl->offsets[w.g] + w.mt * BM, w.ks);
            }
            bulk_commit();
          }
        }
      } else if (ok && warp_live && mine) {
        // through shared memory, so that the stores run along rows: 64 bytes of
        // every row at a time, or where the rows' alignment wants one element a
        // store, as many as there is room for
        constexpr int ELT = EPI == FP8_BF16 || EPI == FP8_GATE_H16 ? 2 : 4;
        const float g = (F32 && p.row_gate != nullptr && vrow) ? p.row_gate[row] : 1.f;
        const int n0 = PAIR ? w.nt * 128 + half * 64 : w.nt * 256 + half * 128;
        const int64_t row_base = ctl->offsets[w.g] + w.mt * BM + q * 32;
        const int nrows = min(32, ctl->offsets[w.g + 1] - static_cast<int>(row_base));
        uint8_t* out = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(w.ks) * p.split_stride * ELT;
        auto piece = [&](int first) { return out_piece<EPI>(acc + first, EPI == FP8_GATE_H16 ? h16_scale : g); };
        if (p.vec_out) {
          constexpr int PER = 64 / ELT;
#pragma unroll
          for (int c = 0; c < 128 / PER; ++c) {
#pragma unroll
            for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(stg + stage_at(lane, v)) = piece(c * PER + v * (16 / ELT));
            __syncwarp();
            const int col = n0 + (PAIR ? c % (64 / PER) : c) * PER;
            if (PAIR && c == 64 / PER) out += p.pair_stride * ELT;  // W3's columns
            const int seg = lane & 3;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = (lane >> 2) + 8 * i;
              if (rr < nrows && col + seg * (16 / ELT) < p.N)
                *reinterpret_cast<uint4*>(out + ((row_base + rr) * p.ld_out + col) * ELT + seg * 16) =
                    *reinterpret_cast<const uint4*>(stg + stage_at(rr, seg));
            }
            __syncwarp();
          }
        } else if (!PAIR) {  // (a cut first projection has N a multiple of 16)
          constexpr int WIDE = G::OUT_BYTES / EPI_WARPS / 32;  // bytes of a row laid out at once
          constexpr int PER = WIDE / ELT, PIECES = WIDE / 16, SWAP = PIECES < 8 ? PIECES - 1 : 7;
          using Word = typename OutWord<ELT>::type;
#pragma unroll
          for (int c = 0; c < 128 / PER; ++c) {
#pragma unroll
            for (int v = 0; v < PIECES; ++v)
              *reinterpret_cast<uint4*>(stg + lane * WIDE + ((v ^ (lane & SWAP)) << 4)) = piece(c * PER + v * (16 / ELT));
            __syncwarp();
            const int col = n0 + c * PER;
#pragma unroll 4
            for (int rr = 0; rr < nrows; ++rr) {
              Word* dst = reinterpret_cast<Word*>(out) + (row_base + rr) * p.ld_out + col;
#pragma unroll
              for (int e0 = 0; e0 < PER; e0 += 32) {
                const int e = e0 + lane;
                if (e < PER && col + e < p.N)
                  dst[e] = *reinterpret_cast<const Word*>(stg + rr * WIDE + (((e * ELT >> 4) ^ (rr & SWAP)) << 4) + (e * ELT & 15));
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (TMA_OUT && storer) bulk_wait();
    if (CLUSTER && !met) { cluster_meet(); cluster_meet(); }
  }
  if (CLUSTER && warp < 4) { cluster_meet(); cluster_meet(); }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- partials
// Thread: four columns of a row (one 16-byte access; the partials' rows are
// padded to whole ones), every partial in order; eight partials' loads in
// flight.
template <bool BF16>
__global__ void __launch_bounds__(128) fp8_reduce_kernel(const Fp8ReduceArgs a) {
  __shared__ int s_last;
  pdl_wait();
  pdl_trigger();
  int64_t r0 = 0, r1 = a.rows;
  if (a.offsets != nullptr) {  // as the product's kernel takes them: clamped, ascending
    if (threadIdx.x == 0) s_last = 0;
    __syncthreads();
    for (int g = threadIdx.x; g <= a.G; g += blockDim.x)
      atomicMax(&s_last, min(max(a.offsets[g], 0), static_cast<int>(a.rows)));
    __syncthreads();
    r0 = min(max(a.offsets[0], 0), static_cast<int>(a.rows));
    r1 = s_last;
  }
  const int c0 = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (c0 >= a.N) return;
  for (int64_t r = r0 + blockIdx.y; r < r1; r += gridDim.y) {
    const float* src = a.P + r * a.ld + c0;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < a.ksplit; k0 += 8) {
      float4 q[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float* s = src + (k0 + u) * a.split_stride;
        q[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + u < a.ksplit) q[u] = *reinterpret_cast<const float4*>(s);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) { v[0] += q[u].x; v[1] += q[u].y; v[2] += q[u].z; v[3] += q[u].w; }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c0 + i < a.N) {
        if (BF16) static_cast<__nv_bfloat16*>(a.out)[r * a.ld_out + c0 + i] = __float2bfloat16(v[i]);
        else static_cast<float*>(a.out)[r * a.ld_out + c0 + i] = v[i];
      }
    }
  }
}

// The hidden activation from a cut first projection: 16 lanes take 128 columns
// of a row, eight each; the partials in order, then as the fused epilogue.
template <bool PAIR>
__global__ void __launch_bounds__(256) fp8_hidden_kernel(const Fp8HiddenArgs a) {
  pdl_wait();
  pdl_trigger();
  const int l = threadIdx.x & 15;
  const int groups = (a.N + 127) >> 7;
  const int rows = min(static_cast<int>(a.rows), *a.total_rows);
  const int64_t items = static_cast<int64_t>(rows) * groups, step = static_cast<int64_t>(gridDim.x) * 16;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  for (int64_t i0 = first & ~int64_t{1}; i0 < items; i0 += step) {  // (both teams of a warp run every step)
    const int64_t i = i0 + (first & 1);
    const int64_t r = i < items ? i / groups : 0;
    const int g = i < items ? static_cast<int>(i - r * groups) : 0;
    const int c = g * 128 + l * 8;
    const bool live = i < items && c < a.N;  // N is a multiple of 16
    float v[8], u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.f;
    if (live) {
      const float* s = a.P + r * a.N + c;
#pragma unroll 4
      for (int k = 0; k < a.ksplit; ++k, s += a.split_stride) {
        const float4 q0 = *reinterpret_cast<const float4*>(s), q1 = *reinterpret_cast<const float4*>(s + 4);
        v[0] += q0.x; v[1] += q0.y; v[2] += q0.z; v[3] += q0.w;
        v[4] += q1.x; v[5] += q1.y; v[6] += q1.z; v[7] += q1.w;
        if (PAIR) {
          const float4 w0 = *reinterpret_cast<const float4*>(s + a.pair_stride);
          const float4 w1 = *reinterpret_cast<const float4*>(s + a.pair_stride + 4);
          u[0] += w0.x; u[1] += w0.y; u[2] += w0.z; u[3] += w0.w;
          u[4] += w1.x; u[5] += w1.y; u[6] += w1.z; u[7] += w1.w;
        }
      }
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = PAIR ? silu_mul(v[j], u[j]) : max_nan(v[j], 0.f);
      m = fmaxf(m, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const Fp8Scale q = fp8_scale(m);
    if (live) {
      *reinterpret_cast<uint2*>(a.H + r * a.N + c) =
          make_uint2(e4m3x4(v[0] * q.inv, v[1] * q.inv, v[2] * q.inv, v[3] * q.inv),
                     e4m3x4(v[4] * q.inv, v[5] * q.inv, v[6] * q.inv, v[7] * q.inv));
      if (l == 0) a.Hs[r * groups + g] = q.scale;
    }
  }
}

// ---------------------------------------------------------------- combine
// Thread: eight columns of a token, all of its rows' 16 bytes in flight.
template <int K>
__global__ void __launch_bounds__(256) fp8_combine_kernel(const Fp8CombineArgs a) {
  pdl_wait();
  pdl_trigger();
  const uint32_t vpr = static_cast<uint32_t>(a.d) >> 3;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;  // T * d < 2^32
  const uint32_t t = i / vpr, v = i - t * vpr;
  if (t >= static_cast<uint64_t>(a.T)) return;
  const int nb = (a.d + 127) >> 7, b = static_cast<int>(v >> 4);
  const uint4* Y = reinterpret_cast<const uint4*>(a.Y);
  uint4 q[K];
  float s[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int64_t row = a.dest_row[static_cast<int64_t>(t) * K + j];
    q[j] = row >= 0 ? __ldcs(Y + row * vpr + v) : make_uint4(0u, 0u, 0u, 0u);
    s[j] = row >= 0 ? a.scales[row * nb + b] : 0.f;
  }
  float acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.f;
  auto add = [&](const uint4& u, float f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[c]));
      acc[2 * c] = fmaf(h.x, f, acc[2 * c]);
      acc[2 * c + 1] = fmaf(h.y, f, acc[2 * c + 1]);
    }
  };
#pragma unroll
  for (int j = 0; j < K; ++j) add(q[j], s[j]);
  for (int e = 0; e < a.n_shared; ++e) {  // shared experts after the routed sum
    const int64_t row = *a.shared_base + e * a.T + t;
    add(Y[row * vpr + v], a.scales[row * nb + b]);
  }
  const int64_t at = static_cast<int64_t>(t) * vpr + v;
  if (a.y_f32 != nullptr) {
    reinterpret_cast<float4*>(a.y_f32)[2 * at] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4*>(a.y_f32)[2 * at + 1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  reinterpret_cast<uint4*>(a.y)[at] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                  pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

// ---------------------------------------------------------------- host
bool map_3d(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint64_t mats, uint64_t ld, uint64_t gs,
            uint32_t box_rows) {
  const uint64_t dims[3] = {K, rows, mats};
  const uint64_t strides[2] = {ld, gs};
  const uint32_t box[3] = {static_cast<uint32_t>(BK), box_rows, 1};
  return make_map_nd(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 3, dims, strides, box);
}

template <int EPI, int AR, bool SB1, bool CLUSTER = false>
cudaError_t launch_t(const Fp8Plan& pl, int num_sms, cudaStream_t s) {
  constexpr size_t bytes = smem_bytes<AR, SB1>();
  static_assert(bytes <= 227 * 1024, "8-bit product: shared memory");
  auto* kernel = fp8_gemm_kernel<EPI, AR, SB1, CLUSTER>;
  const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), static_cast<int>(bytes));
  if (e != cudaSuccess) return e;
  if constexpr (CLUSTER) {
    static_assert(Geo<AR>::STAGES * Geo<AR>::STAGE_BYTES >= (MAX_CLUSTER - 1) * CL_ROWS * CL_LD * 4, "the sums' room");
    // groups of so few rows have one row tile each
    const int64_t tiles = std::min<int64_t>(pl.p.G, pl.p.a_rows) * pl.p.n_tiles;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(tiles * pl.p.cluster)), pl.p.cluster, dim3(NUM_THREADS),
                              bytes, s, pl.a, pl.b0, pl.b1, pl.out, pl.p);
  } else {
    return launch_pdl(kernel, dim3(num_sms), dim3(NUM_THREADS), bytes, s, pl.a, pl.b0, pl.b1, pl.out, pl.p);
  }
}

template <int EPI>
cudaError_t launch_ar(const Fp8Plan& pl, int num_sms, cudaStream_t s) {
  if constexpr (EPI == FP8_BF16 || EPI == FP8_F32) {
    if (pl.p.cluster > 1) return launch_t<EPI, 32, false, true>(pl, num_sms, s);  // (CL_ROWS rows at most)
    if (pl.sb1) return launch_t<EPI, 128, true>(pl, num_sms, s);
  }
  if (pl.ar == 32) return launch_t<EPI, 32, false>(pl, num_sms, s);
  if (pl.ar == 64) return launch_t<EPI, 64, false>(pl, num_sms, s);
  return launch_t<EPI, 128, false>(pl, num_sms, s);
}

}  // namespace

int fp8_ksplit(int64_t rows, int G, int N, int K, bool summed_anyway) {
  // Most 128-row tiles `rows` rows can make over G groups.
  const int64_t g = std::min<int64_t>(G, rows);
  const int64_t tiles = (g + (rows - g) / BM) * ((N + 255) / 256);
  const int64_t num_kb = (K + BK - 1) / BK;
  if (tiles <= 0 || tiles > 4 * kSplitTargetCtas) return 1;
  // Rows count in powers of two, so that the choice is constant between them.
  int64_t r2 = 1;
  while (r2 < rows) r2 <<= 1;
  if (r2 <= 64) {
    // A few rows: the weights' stream is the time, and about 96 CTAs carry what
    // HBM gives (a k-block takes a CTA's loop 0.42 to 0.45 us, 73 GB/s, wherever the
    // weights lie).  One token times 14336 x 4096, 56 tiles: uncut 19.8 us, cut in
    // two 18.2 us, in five 20.7 us, each with the second launch; 224 tiles, two experts' first projections: uncut 52
    // us, cut in three 57 us.  The ranges stay within one wave of CTAs: 86 tiles
    // (one token times 22016 x 4096) cut in two, 172 ranges, take 27.4 us, uncut 20.7.
    // Where a launch that follows sums the partials anyway, a cut is free, and
    // fills the SMs (one token's second projections, 32 tiles: three ranges 30.0 us,
    // four 29.4 us).
    if (!summed_anyway && tiles >= 96) return 1;
    const int64_t wave = std::max<int64_t>(kSplitTargetCtas / tiles, 1);
    const int64_t want = summed_anyway ? wave : std::min((96 + tiles - 1) / tiles, wave);
    const int64_t ks = std::min(want, std::max<int64_t>(num_kb / 2, 1));
    const int64_t per = (num_kb + ks - 1) / ks;
    return static_cast<int>((num_kb + per - 1) / per);
  }
  // Time of a cut, in tenths of a k-block's: the longest CTA runs ceil(units /
  // SMs) ranges of `per` k-blocks, each followed by an epilogue of about 5
  // k-blocks' time; every partial is written and read once more (a k-block's
  // time moves 2.7 MB), and a cut product needs a second launch (8).
  const int64_t epi = 50, launch = 80;
  int64_t best = 1, best_t = (tiles + kSplitTargetCtas - 1) / kSplitTargetCtas * (10 * num_kb + epi);
  // (More ranges than two waves of CTAs, or sixteen of many tiles, gain under a tenth in this sum.)
  const int64_t most = std::min<int64_t>(num_kb / 2, std::max<int64_t>(16, 2 * kSplitTargetCtas / tiles));
  for (int64_t ks = 2; ks <= most; ++ks) {
    const int64_t per = (num_kb + ks - 1) / ks;
    const int64_t ranges = (num_kb + per - 1) / per;
    const int64_t t = (tiles * ranges + kSplitTargetCtas - 1) / kSplitTargetCtas * (10 * per + epi) +
                      r2 * N * ranges / 34000 + launch;
    if (t * 32 < best_t * 31) { best = ranges; best_t = t; }
  }
  return static_cast<int>(best);
}

int fp8_cluster(int64_t rows, int ksplit, int K, int b_rows) {
  // 8 rows, 14336 x 4096 in two ranges: 13.1 us, by partials and a second launch 15.3
  // us; 2048 x 768 in three: 6.5 and 8.3 us (weights in L2).  16 rows tie, and
  // 64 rows' sums take an SM 4 us to receive.  More ranges than a cluster has
  // CTAs pay for their second launch from about three k-blocks less a range on
  // (2048 x 4096, 12 ranges of 3 or 8 of 4: 9.0 and 8.7 us; 768 x 8192, 32 of 2
  // or 8 of 8: 9.8 and 10.1 us).
  if (rows > CL_ROWS || b_rows == 1 || ksplit < 2) return 1;
  const int num_kb = (K + BK - 1) / BK, c = std::min(ksplit, MAX_CLUSTER);
  const int per = (num_kb + c - 1) / c, per_cut = (num_kb + ksplit - 1) / ksplit;
  return per <= per_cut + 3 ? (num_kb + per - 1) / per : 1;
}

cudaError_t plan_fp8(const Fp8Args& g, Fp8Plan* pl, const char** why) {
  *why = nullptr;
  const bool pair = g.epi == FP8_SWIGLU || g.epi == FP8_PAIR_F32;
  if (g.epi == FP8_GATE_H16 && (g.max_group_rows <= 64 || g.b_rows == 1 || g.row_gate == nullptr)) {
    *why = "8-bit product: the fp16 epilogue takes whole tiles and a gate";
    return cudaErrorInvalidValue;
  }
  pl->epi = g.epi;
  pl->sb1 = g.b_rows == 1;
  pl->ar = pl->sb1 ? 128 : g.max_group_rows <= 32 ? 32 : g.max_group_rows <= 64 ? 64 : 128;
  const uint64_t ad[2] = {static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.a_rows)};
  const uint64_t as[1] = {static_cast<uint64_t>(g.lda)};
  const uint32_t abox[2] = {static_cast<uint32_t>(BK), static_cast<uint32_t>(pl->ar)};
  const uint64_t K = g.K, N = g.N, G = g.G, ldb = g.ldb, gsb = g.gsb;
  if (!make_map_nd(&pl->a, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.A, 2, ad, as, abox) || !map_3d(&pl->b0, g.B0, K, N, G, ldb, gsb, pair ? 128 : 256) ||
      (pair && !map_3d(&pl->b1, g.B1, K, N, G, ldb, gsb, 128))) {
    *why = "cuTensorMapEncodeTiled failed (alignment or driver entry point)";
    return cudaErrorInvalidValue;
  }
  if (!pair) pl->b1 = pl->b0;  // (not read)
  Fp8Params& p = pl->p;
  p.G = g.G;
  p.N = g.N;
  const int bn = pair ? 128 : 256;
  p.n_tiles = (g.N + bn - 1) / bn;
  p.num_kb = (g.K + BK - 1) / BK;
  p.ksplit = g.epi == FP8_F32 || g.epi == FP8_PAIR_F32 ? std::max(1, std::min(g.ksplit, p.num_kb)) : 1;
  p.cluster = std::max(1, g.cluster);
  if (p.cluster > 1) p.ksplit = p.cluster;
  p.kb_per = (p.num_kb + p.ksplit - 1) / p.ksplit;
  p.a_rows = g.a_rows;
  p.sa = g.sa;
  p.sa_ld = g.sa_ld;
  p.sb0 = g.sb0;
  p.sb1 = g.sb1;
  p.sb_gs = static_cast<int64_t>(pl->sb1 ? g.N : (g.N + 127) / 128) * p.num_kb;
  p.out = g.out;
  p.ld_out = g.ld_out;
  p.split_stride = g.split_stride;
  p.pair_stride = g.pair_stride;
  p.out_scales = g.out_scales;
  const int elt = g.epi == FP8_BF16 || g.epi == FP8_GATE_H16 ? 2 : 4;
  // (a partial's rows have room behind N for the last piece)
  const bool whole_n = g.epi == FP8_F32 && p.ksplit > 1 && p.cluster == 1 && g.ld_out >= (g.N + 3) / 4 * 4;
  p.vec_out = ((reinterpret_cast<uintptr_t>(g.out) | static_cast<uintptr_t>(g.ld_out * elt) |
                static_cast<uintptr_t>(whole_n ? 0 : static_cast<int64_t>(g.N) * elt) | static_cast<uintptr_t>(g.split_stride * elt) |
                static_cast<uintptr_t>(g.pair_stride * elt)) & 15) == 0;
  // whole tiles of the output by TMA, where its rows allow it (a store is cut off at
  // the row's end in whole 16-byte pieces only)
  const bool act = g.epi == FP8_SWIGLU || g.epi == FP8_RELU;
  const int oelt = act ? 1 : elt;
  p.tma_out = 0;
  pl->out = pl->a;
  if (pl->ar == 128 && g.epi != FP8_PAIR_F32 &&
      ((reinterpret_cast<uintptr_t>(g.out) | static_cast<uintptr_t>(g.ld_out * oelt) |
        static_cast<uintptr_t>(whole_n ? 0 : static_cast<int64_t>(g.N) * oelt) | static_cast<uintptr_t>(g.split_stride * oelt)) & 15) == 0) {
    const CUtensorMapDataType type = act ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                         : g.epi == FP8_GATE_H16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                         : elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const uint64_t od[3] = {N, static_cast<uint64_t>(g.a_rows), static_cast<uint64_t>(p.ksplit)};
    const uint64_t os[2] = {static_cast<uint64_t>(g.ld_out) * oelt,
                            static_cast<uint64_t>(p.ksplit > 1 ? g.split_stride : g.a_rows * g.ld_out) * oelt};
    const uint32_t obox[3] = {static_cast<uint32_t>(128 / oelt), 128, 1};
    p.tma_out = make_map_nd(&pl->out, type, g.out, 3, od, os, obox);
  }
  p.row_gate = g.row_gate;
  p.offsets = g.offsets;
  p.err = g.err;
  p.limit_ns = kWaitLimitNs;
  return cudaSuccess;
}

cudaError_t launch_fp8(const Fp8Plan& pl, int num_sms, cudaStream_t s) {
  switch (pl.epi) {
    case FP8_BF16: return launch_ar<FP8_BF16>(pl, num_sms, s);
    case FP8_F32: return launch_ar<FP8_F32>(pl, num_sms, s);
    case FP8_GATE_H16: return launch_t<FP8_GATE_H16, 128, false>(pl, num_sms, s);
    case FP8_PAIR_F32: return launch_ar<FP8_PAIR_F32>(pl, num_sms, s);
    case FP8_SWIGLU: return launch_ar<FP8_SWIGLU>(pl, num_sms, s);
    default: return launch_ar<FP8_RELU>(pl, num_sms, s);
  }
}

cudaError_t launch_fp8_reduce(const Fp8ReduceArgs& a, cudaStream_t s) {
  if (a.rows <= 0 || a.N <= 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((a.N + 511) / 512), static_cast<unsigned>(std::min<int64_t>(a.rows, 65535)));
  return a.out_is_bf16 ? launch_pdl(fp8_reduce_kernel<true>, grid, dim3(128), 0, s, a)
                       : launch_pdl(fp8_reduce_kernel<false>, grid, dim3(128), 0, s, a);
}

cudaError_t launch_fp8_hidden(const Fp8HiddenArgs& a, int num_sms, cudaStream_t s) {
  const int64_t items = a.rows * ((a.N + 127) / 128);
  if (items <= 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + 15) / 16, num_sms * 8)));
  return a.pair_stride > 0 ? launch_pdl(fp8_hidden_kernel<true>, grid, dim3(256), 0, s, a)
                           : launch_pdl(fp8_hidden_kernel<false>, grid, dim3(256), 0, s, a);
}

cudaError_t launch_fp8_combine(const Fp8CombineArgs& a, cudaStream_t s) {
  const uint64_t n = static_cast<uint64_t>(a.T) * (a.d / 8);  // below 2^29
  if (n == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256));
  switch (a.k) {
    case 1: return launch_pdl(fp8_combine_kernel<1>, grid, dim3(256), 0, s, a);
    case 2: return launch_pdl(fp8_combine_kernel<2>, grid, dim3(256), 0, s, a);
    case 3: return launch_pdl(fp8_combine_kernel<3>, grid, dim3(256), 0, s, a);
    case 4: return launch_pdl(fp8_combine_kernel<4>, grid, dim3(256), 0, s, a);
    case 5: return launch_pdl(fp8_combine_kernel<5>, grid, dim3(256), 0, s, a);
    case 6: return launch_pdl(fp8_combine_kernel<6>, grid, dim3(256), 0, s, a);
    case 7: return launch_pdl(fp8_combine_kernel<7>, grid, dim3(256), 0, s, a);
    default: return launch_pdl(fp8_combine_kernel<8>, grid, dim3(256), 0, s, a);
  }
}

}  // namespace moe
