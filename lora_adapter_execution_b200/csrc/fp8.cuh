// The 8-bit frozen base: the quantiser of blocks of 128 and the block-scaled
// product on the tensor cores, with the adapters' K blocks in the same kernel.
//
// Quantiser. A block (1 x 128 of a row, 128 x 128 of a weight) is held as
// e4m3 values q and one scale s, the smallest power of two >= amax / 448 (448 is
// e4m3's largest value), at least 2^-126; 1 for a block of zeros; NaN for a block
// that holds an infinity or a NaN, so that whatever reads the block is NaN.
// x / s is exact in fp32 (a power of two), so the one rounding is the one to
// e4m3 (nearest, ties to even), and |x / s| <= 448: nothing saturates.
//
// Product. Y[t, n] = sum over K blocks b of Sx[b, t] · Sw[b, n / 128] · (sum over k
// in b of Xq[t, k] · Wq[k, n]). The scales differ per row and per block, so they
// cannot wait for the end of the contraction: each K block's 128 x BN product goes
// to its own TMEM buffer, and warps add it, scaled, to fp32 accumulators they
// keep in registers, while the tensor cores fill the next buffer.
#pragma once

#include "common.cuh"
#include "gemm.cuh"
#include "internal.h"

namespace lora {

// ------------------------------------------------------------------ quantiser
constexpr int kQBlock = 128;

// Scale of a block from the largest bf16 magnitude in it (bits without the sign).
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F80u) return __uint_as_float(0x7FC00000u);  // inf or NaN in the block
  if (amax_bits == 0) return 1.0f;
  // amax = m · 2^e, 1 <= m < 2 (subnormals: e < -126, clamped below); 448 = 1.75 · 2^8
  const int e = static_cast<int>(amax_bits >> 7) - 127;
  const int s = e - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);  // 0x60: m = 1.75
  return __uint_as_float(static_cast<uint32_t>(max(s, -126) + 127) << 23);
}
// 1 / s of such a scale (exact: s is a power of two, 2^-126 .. 2^120, or NaN)
__device__ __forceinline__ float fp8_inverse(float s) {
  const uint32_t b = __float_as_uint(s);
  return b >= 0x7F800000u ? s : __uint_as_float((254u - (b >> 23)) << 23);
}
__device__ __forceinline__ uint32_t fp8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// 8 bf16 (one 16-byte load) as e4m3 of x · inv
__device__ __forceinline__ uint2 fp8_pack8(const uint4 &v, float inv) {
  uint2 o;
  o.x = fp8_pack2(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv) | (fp8_pack2(bf16_lo(v.y) * inv, bf16_hi(v.y) * inv) << 16);
  o.y = fp8_pack2(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv) | (fp8_pack2(bf16_lo(v.w) * inv, bf16_hi(v.w) * inv) << 16);
  return o;
}
// largest magnitude of 8 bf16, as bits (monotone: inf 0x7F80 and NaNs above all numbers)
__device__ __forceinline__ uint32_t fp8_amax8(const uint4 &v) {
  // the two halves of each word apart: __vmaxu2 is the packed unsigned maximum
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(a & 0xFFFFu, a >> 16);
}

constexpr int kQRowsCols = 1024;  // columns of a warp's piece of a row: 4 loads of 16 bytes per lane
constexpr int kQRowsWarps = 8;

// Rows in blocks of 1 x 128: Q[i] = e4m3(X[perm[i]] / s) (perm null: i), scale of
// block b of row i at S[b * T + i]; Xs, if given, receives the row itself (the plan's
// sorted copy, for one read of X). A warp takes 1024 columns of one row, a half-warp
// one block per load; a CTA's 8 warps take 8 rows in turn, so that their scales fill
// one 32-byte sector. d % 16 == 0. Bound by HBM (3 bytes an element, 5 with the copy):
// 8192 x 11008 in 48 us, 88 % of the measured copy rate (one 16-byte load at a time
// per thread, with 64-bit divisions: 99 us).
__global__ void __launch_bounds__(32 * kQRowsWarps)
    lora_fp8_rows_kernel(const uint16_t *__restrict__ X, const int32_t *__restrict__ perm, int64_t T, int64_t d,
                         uint8_t *__restrict__ Q, float *__restrict__ S, uint16_t *__restrict__ Xs) {
  pdl_wait();
  pdl_launch_dependents();  // the next kernel may set itself up meanwhile (never before the last one is done)
  const int lane = threadIdx.x & 31;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kQRowsCols + lane * 8;
  for (int64_t i = static_cast<int64_t>(blockIdx.y) * kQRowsWarps + (threadIdx.x >> 5); i < T;
       i += static_cast<int64_t>(gridDim.y) * kQRowsWarps) {
    const uint16_t *x = X + (perm ? __ldg(perm + i) : i) * d;
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v[u] = c0 + 256 * u < d ? __ldg(reinterpret_cast<const uint4 *>(x + c0 + 256 * u)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t c = c0 + 256 * u;
      uint32_t a = fp8_amax8(v[u]);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      if (c < d) {
        const float s = fp8_scale(a);
        *reinterpret_cast<uint2 *>(Q + i * d + c) = fp8_pack8(v[u], fp8_inverse(s));
        if (Xs) *reinterpret_cast<uint4 *>(Xs + i * d + c) = v[u];
        if ((lane & 15) == 0) S[(c / kQBlock) * T + i] = s;
      }
    }
  }
}

// Up to three arrays' rows into the plan's order in one launch: 16-byte pieces of X and
// of the keep bits (either may be absent), and U's rows padded with zeros to rp columns.
__global__ void __launch_bounds__(256)
    lora_gather_set_kernel(const int32_t *__restrict__ perm, int64_t T, const uint4 *__restrict__ X, uint4 *Xs,
                           int x_row, const uint4 *__restrict__ B, uint4 *Bs, int b_row, const float *__restrict__ U,
                           float *Us, int r, int rp) {
  pdl_wait();
  pdl_launch_dependents();
  // a warp per row
  const int lane = threadIdx.x & 31;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < T; i += nw) {
    const int64_t src = perm ? __ldg(perm + i) : i;
    if (X) {
      for (int c = lane; c < x_row; c += 128) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + 32 * u < x_row) v[u] = __ldg(X + src * x_row + c + 32 * u);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + 32 * u < x_row) Xs[i * x_row + c + 32 * u] = v[u];
      }
    }
    if (B)
      for (int c = lane; c < b_row; c += 32) Bs[i * b_row + c] = __ldg(B + src * b_row + c);
    for (int c = lane; c < rp; c += 32) Us[i * rp + c] = c < r ? __ldg(U + src * r + c) : 0.f;
  }
}

// A weight in blocks of 128 x 128: one CTA per block, the block in registers
// (8 loads of 16 bytes per thread) between its maximum and its values. Scale of
// block (i, j) at S[i * ceil(cols / 128) + j]. Bound by HBM: 4096 x 11008 in 22.4 us,
// 94 % of the measured copy rate.
__global__ void __launch_bounds__(256)
    lora_fp8_weight_kernel(const uint16_t *__restrict__ W, int64_t rows, int64_t cols, uint8_t *__restrict__ Q,
                           float *__restrict__ S) {
  __shared__ uint32_t wmax[8];
  const int64_t nb = (cols + kQBlock - 1) / kQBlock;
  const int64_t bi = blockIdx.x / nb, bj = blockIdx.x % nb;
  const int64_t col = bj * kQBlock + (threadIdx.x & 15) * 8;
  const int64_t row0 = bi * kQBlock + (threadIdx.x >> 4);
  uint4 v[8];
  uint32_t a = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t r = row0 + 16 * u;
    v[u] = (col < cols && r < rows) ? __ldg(reinterpret_cast<const uint4 *>(W + r * cols + col))
                                    : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) a = max(a, fp8_amax8(v[u]));
  a = __reduce_max_sync(0xFFFFFFFFu, a);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
  __syncthreads();
  a = wmax[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) a = max(a, wmax[w]);
  const float s = fp8_scale(a);
  const float inv = fp8_inverse(s);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t r = row0 + 16 * u;
    if (col < cols && r < rows) *reinterpret_cast<uint2 *>(Q + r * cols + col) = fp8_pack8(v[u], inv);
  }
  if (threadIdx.x == 0) S[blockIdx.x] = s;
}

// ------------------------------------------------------------------ product
// 12 warps: 0 copies A, W and the adapter blocks, 1 and 2 issue the MMAs (1 owns
// TMEM), 3 is the fix-up warp of adapter blocks (as in gemm.cuh), and two
// warpgroups accumulate: thread = output row (a TMEM lane), warpgroup h = columns
// [h·BN/2, (h+1)·BN/2) of the tile, so at BN = 256 each meets one weight block per
// K block. Two issuing warps, because two waits, four MMAs and two commits took one
// about 1,100 cycles a block beside everything else: warp 1 + e takes the stages of
// parity e and fills TMEM buffers of its own. A tile's adapter blocks therefore end
// in up to two buffers (those on even stages, those on odd ones), drained before
// the base blocks'. What bounds it: a block of 128 takes about 1070 cycles (5003 x
// 11008 x 4096 under ncu: 461,182 for the longest CTA's five tiles of 86 blocks), its
// MMAs 512 of them. Loads alone, free-running (4 stages of 48 KB), took 760, the
// hand-over of the buffers alone 608: they add up more than they overlap. Which of the
// path from L2 (39 bytes a cycle and SM are reached) and the shared memory port holds
// the loads was not measured. And tiles come in whole rounds: 640 of them on 148 CTAs
// are five rounds for 4.32 (592 tiles, four rounds: 232 us, 640: 290). 5003 x 11008 x 4096:
// 268 us under ncu, 1.69 PFLOP/s, 285 in a graph over three sets of operands (one issuing
// warp, scales loaded a block ahead: a third slower; a pair of CTAs on 256 rows,
// cta_group::2: 5 % slower).
//
// The adapters' s·U (s·dU) comes as two bf16 parts, hi + lo, 16 bits (the image that
// lora_shrink_kernel writes for the bf16 layer, too): a third part would make half as
// many adapter blocks again. What it costs before the rounding to bf16 is 2.3e-6 of the
// output's norm (the fleet's dX; measured against 64 bits), where that rounding itself
// is 1.7e-3: one output in 700 becomes its bf16 neighbour.
constexpr int kF8Groups = 2;                   // accumulating warpgroups
constexpr int kF8Sum = 128 * kF8Groups;        // accumulating threads
constexpr int kF8Threads = 128 + kF8Sum;
constexpr int kF8K = 128;  // bytes (= elements) of K per stage: one scale block, one swizzle row
constexpr int kF8StageA = kBM * kF8K;  // 16 KB; an adapter block's s·U image has the same size
// Registers a thread at BN = 256 after the split: what the copying warps give up
// covers what the accumulating ones take (the launch's 168 per thread).
constexpr int kF8RegsCopy = 64, kF8RegsSum = 216;
static_assert(128 * kF8RegsCopy + kF8Sum * kF8RegsSum <= 168 * kF8Threads, "register split");
// K blocks whose scales a thread has on their way (cp.async into slots of its
// own, so no barrier). Under the operands' load an L2 access takes several
// thousand cycles: 3 blocks ahead cost a tenth of the time (5003 x 11008 x 4096:
// 310 us, 278 us with 15 ahead).
constexpr int kScaleAhead = 16;
template <int BN>
struct F8 {
  static constexpr int kStageB = BN * kF8K;
  static constexpr int kStage = kF8StageA + kStageB;
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kBuf = BN == 256 ? 2 : 4;       // TMEM buffers (512 columns in all)
  static constexpr int kCols = BN / kF8Groups;         // columns per accumulating thread
  static constexpr int kSlot = (BN / 64) * 16 * 128;   // one 16-row slice of B_pool over the tile's columns
  static constexpr int kBars = 512;
  // scales on their way to the accumulating threads: [kScaleAhead][threads]
  static constexpr int kScales = kScaleAhead * kF8Sum * 4;
  static constexpr int kSmem = 1024 + kStages * kStage + kBars + kScales;
};
static_assert(F8<128>::kStages % 2 == 0 && F8<256>::kStages % 2 == 0, "a stage belongs to one issuing warp");
static_assert(kF8StageA == kAugBlockBytes, "an adapter block's image fills the A half of a stage");
static_assert(F8<128>::kStages * F8<128>::kStage >= kBM * 128 * 4, "split-K exchange must fit the stage ring");
static_assert(F8<256>::kStages * F8<256>::kStage >= kBM * 256 * 4, "split-K exchange must fit the stage ring");

// A position in a ring of N buffers and its phase.
template <int N>
struct F8Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};
struct Fp8Params {
  GemmParams g;     // geometry, plan tables, output and mask (a_sorted: A rows are in the plan's order)
  const float *Sx;  // [K blocks][T]: scale of A's row i (in A's row order) in K block b
  const float *Sw;  // scale of weight block (K block b, column block j) at b * sw_k + j * sw_n
  int32_t sw_k, sw_n, n_nb;  // n_nb: column blocks
  int32_t a_bytes;  // bytes of an A copy: the whole tile, or only the rows that a short batch has
                    // (the other rows' products are whatever the stage held, and are not used)
};

// D[tmem] (+)= A·B, e4m3 operands, fp32 accumulation, K = 32.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 consecutive fp32 columns of this thread's TMEM lane, waited for (one statement,
// so that nothing that uses them can move before the wait).
__device__ __forceinline__ void tmem_ld32w(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4 with e4m3 A/B (format 0) and fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// 4 bytes from global to this thread's shared slot, or zero when bytes is 0.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)::"memory");
  return r != 0;
}
// Every thread of the CTA meets here once, from either branch of the kernel.
__device__ __forceinline__ void f8_join() { asm volatile("barrier.sync 0, %0;" ::"n"(kF8Threads) : "memory"); }

// B_KMAJOR: W read as its own rows [N, K] (the backward's W^T); otherwise [K, N],
// N contiguous (MN-major). DROP: the adapter term is masked (backward, dropout).
// The K split (p.ksplit > 1) is for BN = 128 only. At BN = 256 the accumulating
// warps hold 128 sums each and take registers from the others (setmaxnreg), so
// the two branches share no code after that point.
template <bool B_KMAJOR, int BN, bool DROP>
__global__ void __launch_bounds__(kF8Threads, 1)
    lora_fp8_gemm_kernel(const __grid_constant__ CUtensorMap mapA,   // A rows, box {128, 128}
                         const __grid_constant__ CUtensorMap mapB,   // W: K-major box {128, BN}; MN-major box {128, 128}
                         const __grid_constant__ CUtensorMap mapBl,  // adapter rows, box {64, 16(, BN/64)}
                         const __grid_constant__ Fp8Params fp) {
  using C = F8<BN>;
  const GemmParams &p = fp.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t stage0 = smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kStages * C::kStage);
  const uint32_t full0 = smem_u32(bars);              // [kStages]
  const uint32_t empty0 = full0 + 8 * C::kStages;     // [kStages]
  const uint32_t fixed0 = empty0 + 8 * C::kStages;    // [kStages] released by the fix-up warp
  const uint32_t accf0 = fixed0 + 8 * C::kStages;     // [kBuf]
  const uint32_t acce0 = accf0 + 8 * C::kBuf;         // [kBuf]
  const uint32_t done0 = acce0 + 8 * C::kBuf;         // [2] after a wait gave up: an issuing warp's MMAs are done
  uint32_t *words = reinterpret_cast<uint32_t *>(bars + 3 * C::kStages + 2 * C::kBuf + 2);
  uint32_t *tmem_slot = words;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(words + 1);
  volatile uint32_t *filled = words + 2;                 // where the copying thread ended: its phase · kStages + its stage
  volatile uint32_t *bmap = words + 3;                   // [kStages] slot of each K step of an adapter block
  volatile uint32_t *bvalid = words + 3 + C::kStages;    // [kStages] AugBlockDesc::valid | nslot << 20
  static_assert((3 * C::kStages + 2 * C::kBuf + 2) * 8 + (3 + 2 * C::kStages) * 4 <= C::kBars, "barrier block");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(fixed0 + 8 * s, 1);
    }
    for (int b = 0; b < C::kBuf; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, kF8Sum / 32);  // one arrival per accumulating warp
    }
    mbar_init(done0, 1);
    mbar_init(done0 + 8, 1);
    *abort_flag = 0;
    *filled = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // Every operand may come from the kernel before this one. The next kernel is not let
  // in early: lora_gemm_kernel reads its W before it waits, and W may be this output.
  pdl_wait();

  const int n_tiles = p.n_mt * p.n_nt;
  const int KB = (p.K + kF8K - 1) / kF8K;
  const bool has_plan = p.tiles != nullptr;
  auto tile_desc = [&](int mt) -> TileDesc { return has_plan ? p.tiles[mt] : regular_tile(mt, p.T); };
  const int S = BN == 128 ? p.ksplit : 1;
  const int q = S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile0 = static_cast<int>(blockIdx.x) / S;
  const int tile_step = S > 1 ? n_tiles : static_cast<int>(gridDim.x);
  // After a wait gave up (every warp has joined): what is in flight ends, each wait
  // bounded too, before TMEM is freed and shared memory given up.
  auto settle = [&]() {
    if (warp == 1 || warp == 2) {
      if (elect_one()) umma_commit(done0 + 8 * (warp - 1));
      __syncwarp();
    }
    if (warp == 1) {
      mbar_wait(done0, 0);
      mbar_wait(done0 + 8, 0);
      __syncwarp();
    }
    if (threadIdx.x == 0) {
      // the last copy into each stage: in this phase before the stage where the copying
      // ended, in the one before from there on (never filled: that phase counts as done)
      const uint32_t end = *filled % C::kStages, ph = *filled / C::kStages;
      for (uint32_t s = 0; s < C::kStages; ++s) mbar_wait(full0 + 8 * s, s < end ? ph : ph ^ 1);
    }
  };

  if (warp < 4) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8RegsCopy));
    if (warp == 0) {
      // ------------------------------------------------ copies: A, W, adapter blocks
      if (lane == 0) {
        prefetch_tmap(&mapA);
        prefetch_tmap(&mapB);
        int stage = 0;
        uint32_t phase = 0;
        int tile;
        for (int k = 0; !*abort_flag && cta_tile(p, k, tile0, tile_step, n_tiles, tile); ++k) {
          int mt, nt;
          tile_coords(tile, p, mt, nt);
          const TileDesc td = tile_desc(mt);
          const int n0 = nt * BN;
          const BlockRange br = block_range(KB, (td.kaug + kAugBlock - 1) / kAugBlock, q, S);
          const int nblk = br.count();
          for (int i = 0; i < nblk; ++i) {
            const int blk = br.block(i, KB);
            if (!mbar_wait(empty0 + 8 * stage, phase ^ 1)) { *abort_flag = 1; break; }
            const uint32_t a_dst = stage0 + stage * C::kStage;
            const uint32_t b_dst = a_dst + kF8StageA;
            const uint32_t fb = full0 + 8 * stage;
            if (blk < KB) {
              mbar_arrive_expect_tx(fb, static_cast<uint32_t>(fp.a_bytes) + C::kStageB);
              tma_load_2d(a_dst, &mapA, fb, blk * kF8K, td.row0);
              if (B_KMAJOR) {
                tma_load_2d(b_dst, &mapB, fb, blk * kF8K, n0);
              } else {
                for (int j = 0; j < BN / 128; ++j)
                  tma_load_2d(b_dst + j * 16384, &mapB, fb, n0 + j * 128, blk * kF8K);
              }
            } else {
              const AugBlockDesc *ab = p.augblocks + td.aug0 + (blk - KB);
              const int4 prow = __ldg(reinterpret_cast<const int4 *>(ab));
              const int info = __ldg(&ab->info);
              const int nslot = info & 15;
              bmap[stage] = static_cast<uint32_t>(info >> 4) & 0xFFu;
              bvalid[stage] = static_cast<uint32_t>(__ldg(&ab->valid)) | (static_cast<uint32_t>(nslot) << 20);
              mbar_arrive_expect_tx(fb, kF8StageA + nslot * C::kSlot);
              bulk_g2s(a_dst, p.uimg + td.uofs + static_cast<int64_t>(blk - KB) * kAugBlockBytes, kAugBlockBytes, fb);
              const int prow_s[4] = {prow.x, prow.y, prow.z, prow.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                if (u < nslot) {
                  if (p.b3d) {
                    tma_load_3d(b_dst + u * C::kSlot, &mapBl, fb, 0, prow_s[u], n0 / 64);
                  } else {
                    for (int j = 0; j < BN / 64; ++j)
                      tma_load_2d(b_dst + u * C::kSlot + j * 2048, &mapBl, fb, n0 + j * 64, prow_s[u]);
                  }
                }
              }
            }
            if (++stage == C::kStages) { stage = 0; phase ^= 1; }
          }
        }
        *filled = phase * C::kStages + stage;
      }
    } else if (warp == 3) {
      // ------------------------------------------------ fix-up (see gemm.cuh): with a
      // plan every stage reaches the MMAs through this warp, which zeroes the rows
      // of an adapter block's slices that belong to another adapter
      if (has_plan) {
        int stage = 0;
        uint32_t phase = 0;
        int tile;
        for (int k = 0;; ++k) {
          const bool go = !*abort_flag && cta_tile(p, k, tile0, tile_step, n_tiles, tile);
          if (!__shfl_sync(0xFFFFFFFFu, go ? 1 : 0, 0)) break;
          int mt, nt;
          tile_coords(tile, p, mt, nt);
          const BlockRange br = block_range(KB, (p.tiles[mt].kaug + kAugBlock - 1) / kAugBlock, q, S);
          const int nblk = br.count();
          bool ok = true;
          for (int i = 0; i < nblk; ++i) {
            const int blk = br.block(i, KB);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(full0 + 8 * stage, phase))) {
              if (lane == 0) *abort_flag = 1;
              ok = false;
              break;
            }
            if (blk >= KB) {
              const uint32_t vw = bvalid[stage];
              const int nsl = static_cast<int>(vw >> 20);
              uint8_t *bsp = smem + stage * C::kStage + kF8StageA;
              bool zeroed = false;
              for (int u = 0; u < nsl; ++u) {
                const int v = static_cast<int>((vw >> (5 * u)) & 31u);
                constexpr int kPer = (BN / 64) * 8;  // 16-byte pieces per slice row
                for (int e = lane; e < (16 - v) * kPer; e += 32) {
                  const int r = v + e / kPer;
                  const int j = (e >> 3) % (BN / 64);
                  *reinterpret_cast<uint4 *>(bsp + u * C::kSlot + j * 2048 + r * 128 + (e & 7) * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
                }
                zeroed |= v < 16;
              }
              if (zeroed) fence_proxy_async_smem();  // the MMA reads through the async proxy
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(fixed0 + 8 * stage);
            if (++stage == C::kStages) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
        }
      }
    } else {
      // ------------------------------------------------ MMA issuers (the whole warp
      // runs the loop, one elected lane issues, so descriptors stay in uniform registers)
      constexpr uint32_t kIdesc = idesc_e4m3(kBM, BN, false, !B_KMAJOR);
      constexpr uint32_t kIdescAug = idesc_bf16(kBM, BN, false, true);
      // A K-major, 128-byte rows: 8-row groups 1 KB apart, a K = 32 step 32 bytes on.
      // B K-major likewise; MN-major: 128-column blocks 16 KB apart, 8 K rows 1 KB
      // apart, a K = 32 step 32 rows (4 KB) on.
      const uint64_t adesc0 = sdesc_sw128(stage0, 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(stage0 + kF8StageA, B_KMAJOR ? 16 : 16384, 1024);
      constexpr uint64_t kAStep = 32 >> 4;
      constexpr uint64_t kBStep = B_KMAJOR ? (32 >> 4) : (4096 >> 4);
      const uint32_t ready0 = has_plan ? fixed0 : full0;
      const int e = warp - 1;
      F8Ring<C::kBuf / 2> ring;
      int stage = 0;
      uint32_t phase = 0;
      int tile;
      for (int k = 0;; ++k) {
        const bool go = !*abort_flag && cta_tile(p, k, tile0, tile_step, n_tiles, tile);
        if (!__shfl_sync(0xFFFFFFFFu, go ? 1 : 0, 0)) break;
        int mt, nt;
        tile_coords(tile, p, mt, nt);
        const int kaug = has_plan ? p.tiles[mt].kaug : 0;
        const BlockRange br = block_range(KB, (kaug + kAugBlock - 1) / kAugBlock, q, S);
        const int nblk = br.count(), naug = br.naug();
        bool ok = true;
        for (int i = 0; i < nblk; ++i) {
          if ((stage & 1) != e) {  // the other warp's
            if (++stage == C::kStages) { stage = 0; phase ^= 1; }
            continue;
          }
          const int blk = br.block(i, KB);
          // this warp's adapter blocks of a tile share one buffer, each base block has its own
          const bool first = i < 2 || i >= naug, last = i + 2 >= naug;
          const int buf = e + 2 * ring.slot;
          if ((first && !__all_sync(0xFFFFFFFFu, mbar_wait(acce0 + 8 * buf, ring.phase ^ 1))) ||
              !__all_sync(0xFFFFFFFFu, mbar_wait(ready0 + 8 * stage, phase))) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + buf * BN;
          const uint64_t ad = adesc0 + static_cast<uint64_t>(stage * (C::kStage >> 4));
          if (elect_one()) {
            if (blk < KB) {
              const uint64_t bd = bdesc0 + static_cast<uint64_t>(stage * (C::kStage >> 4));
              umma_e4m3(d_tmem, ad, bd, kIdesc, 0u);
              umma_e4m3(d_tmem, ad + kAStep, bd + kBStep, kIdesc, 1u);
              umma_e4m3(d_tmem, ad + 2 * kAStep, bd + 2 * kBStep, kIdesc, 1u);
              umma_e4m3(d_tmem, ad + 3 * kAStep, bd + 3 * kBStep, kIdesc, 1u);
            } else {
              // bf16 image columns against the slots of B_pool rows, 16 ranks a step
              const int steps = min(4, (kaug - (blk - KB) * kAugBlock) / 16);
              const uint32_t map = bmap[stage];
              const uint32_t b_s = stage0 + stage * C::kStage + kF8StageA;
              for (int u = 0; u < steps; ++u) {
                const uint64_t bd = sdesc_sw128(b_s + ((map >> (2 * u)) & 3u) * C::kSlot, 2048, 1024);
                umma_bf16(d_tmem, ad + u * kAStep, bd, kIdescAug, (i < 2 && u == 0) ? 0u : 1u);
              }
            }
            umma_commit(empty0 + 8 * stage);
            if (last) umma_commit(accf0 + 8 * buf);  // the buffer is complete
          }
          __syncwarp();
          if (last) ring.next();
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
      }
    }
    __syncwarp();
    if constexpr (BN == 256) {
      tc_fence_before();
      f8_join();  // every TMEM read is done
      if (*abort_flag) settle();
      if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
      }
      return;
    }
  } else {
    // -------------------------------------------------- accumulating warps
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8RegsSum));
    const int h = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + h * C::kCols;
    uint32_t rings = 0;  // buffers of even and of odd stages drained so far, a byte each
    int par = 0;                       // parity of the next block's stage
    int tile;
    for (int k = 0; !*abort_flag && cta_tile(p, k, tile0, tile_step, n_tiles, tile); ++k) {
      int mt, nt;
      tile_coords(tile, p, mt, nt);
      const TileDesc td = tile_desc(mt);
      const BlockRange br = block_range(KB, (td.kaug + kAugBlock - 1) / kAugBlock, q, S);
      const bool valid = row < td.rows;
      const int col0 = nt * BN + h * C::kCols;
      int64_t orig = 0;
      if (valid) orig = has_plan ? (td.contig >= 0 ? td.contig + row : p.perm[td.row0 + row]) : td.row0 + row;
      float acc[C::kCols];
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) acc[i] = 0.f;
      // Scales: the row's by cp.async into slots of the thread's own (no barrier),
      // kScaleAhead - 1 K blocks ahead; the weight block's, the same for the warp,
      // 32 K blocks at a time in the lanes of one register.
      const int nb = col0 / kQBlock;
      const bool in = valid && nb < fp.n_nb;
      const uint32_t sc = smem_u32(smem + C::kStages * C::kStage + C::kBars) + (threadIdx.x - 128) * 4;
      const uint32_t sc_bytes = in ? 4u : 0u;  // 0: the slot becomes zero
      const float *sx = in ? fp.Sx + static_cast<int64_t>(br.kb_lo) * p.T + td.row0 + row : fp.Sx;
      const int64_t sx_step = in ? p.T : 0;
      const float *sw = fp.Sw + static_cast<int64_t>(min(nb, fp.n_nb - 1)) * fp.sw_n + static_cast<int64_t>(br.kb_lo) * fp.sw_k;
      auto fetch_scale = [&](int j, int slot) {
        if (j < br.nbase) cp_async4(sc + slot * (kF8Sum * 4), sx, sc_bytes);
        cp_async_commit();
        sx += sx_step;
      };
#pragma unroll
      for (int j = 0; j < kScaleAhead - 1; ++j) fetch_scale(j, j);
      bool ok = true;
      // one complete TMEM buffer of the stages of parity e: each 32 columns handed
      // to `add` as they arrive, the buffer released once all are in registers
      auto drain = [&](int e, auto add) -> bool {
        const uint32_t n = (rings >> (8 * e)) & 0xFFu;
        const int buf = e + 2 * (n % (C::kBuf / 2));
        // (agreed by the warp: what follows is for whole warps)
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(accf0 + 8 * buf, (n / (C::kBuf / 2)) & 1u))) {
          *abort_flag = 1;
          return false;
        }
        tc_fence_after();
        const uint32_t ta = lane_base + buf * BN;
        if (quarter * 32 < td.rows) {  // (a warp without rows has nothing to add)
#pragma unroll
          for (int c = 0; c < C::kCols / 32; ++c) {
            float v[32];
            tmem_ld32w(ta + c * 32, v);
            if (c + 1 == C::kCols / 32) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(acce0 + 8 * buf);
            }
            add(c, v);
          }
        } else if (lane == 0) {
          mbar_arrive(acce0 + 8 * buf);
        }
        // (the count of parity e, modulo a power of two that its byte holds)
        rings = (rings & ~(0xFFu << (8 * e))) | (((n + 1) & 0x7Fu) << (8 * e));
        return true;
      };
      // the adapter term first, as it is or masked: the blocks on this parity's
      // stages, then those on the other's
      const float one = DROP ? p.inv_keep : 1.f;
      const int naug = br.naug();
#pragma unroll 1
      for (int u = 0; ok && u < min(naug, 2); ++u) {
        ok = drain(par ^ u, [&](int c, const float (&v)[32]) {
          if constexpr (DROP) {
            const int cc = col0 + c * 32;
            uint32_t keep = 0;
            if (valid && cc < p.N)
              keep = p.keep_bits ? __ldg(p.keep_bits + orig * p.wpr + (cc >> 5))
                                 : keep_mask32(p.seed, p.thr, static_cast<uint64_t>(orig * p.N + cc));
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c * 32 + i] += ((keep >> i) & 1u) ? one * v[i] : 0.f;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c * 32 + i] += v[i];
          }
        });
      }
      par ^= naug & 1;
      float sw_lane = 0.f;
#pragma unroll 1
      for (int j = 0; ok && j < br.nbase; ++j) {
        if ((j & 31) == 0) sw_lane = j + lane < br.nbase ? __ldg(sw + static_cast<int64_t>(j + lane) * fp.sw_k) : 0.f;
        cp_async_wait<kScaleAhead - 2>();
        const float s = ld_shared_f32(sc + (j % kScaleAhead) * (kF8Sum * 4)) * __shfl_sync(0xFFFFFFFFu, sw_lane, j & 31);
        fetch_scale(j + kScaleAhead - 1, (j + kScaleAhead - 1) % kScaleAhead);
        ok = drain(par, [&](int c, const float (&v)[32]) {
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c * 32 + i] = fmaf(s, v[i], acc[c * 32 + i]);
        });
        par ^= 1;
      }
      if (!ok) break;
      if (S == 1) {
        if (valid) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + orig * p.N + col0);
#pragma unroll
          for (int j = 0; j < C::kCols / 8; ++j) {
            if (col0 + 8 * j < p.N) {
              const float *a = acc + 8 * j;
              dst[j] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                                  pack_bf16x2(a[6], a[7]));
            }
          }
        }
      } else if (quarter * 32 < td.rows) {
        // split-K: this CTA's partial sums into its stage ring (its MMAs are done:
        // their last buffer was just read), column by column, rows contiguous.
        // Generic writes after the ring's async-proxy writes, which completed on
        // the full barriers before the MMAs ran.
        float *x = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int i = 0; i < C::kCols; ++i) x[(h * C::kCols + i) * kBM + row] = acc[i];
      }
    }
    if constexpr (BN == 256) {
      tc_fence_before();
      f8_join();
      return;
    }
  }

  if constexpr (BN == 128) {
    tc_fence_before();
    f8_join();
    if (*abort_flag) settle();
    if (warp == 1) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem_base, 512);
    }
    if (S > 1) {
      // CTA q of the cluster sums and stores columns [q·BN/S, (q+1)·BN/S), the ranks
      // in order (the result does not depend on timing): one thread per row and 8
      // columns
      cluster_barrier();
      if (tile0 < n_tiles && !*abort_flag) {
        int mt, nt;
        tile_coords(tile0, p, mt, nt);
        const TileDesc td = tile_desc(mt);
        const int width = BN / S;
        const int rpad = (td.rows + 31) & ~31;
        const int items = rpad * (width / 8);
        for (int e = threadIdx.x; e < items; e += kF8Threads) {
          const int row = e % rpad;
          const int cc = q * width + (e / rpad) * 8;
          const int col = nt * BN + cc;
          if (row < td.rows && col < p.N) {
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = 0.f;
            for (int src = 0; src < S; ++src) {
              const uint32_t a =
                  map_rank(stage0 + static_cast<uint32_t>((cc * kBM + row) * 4), static_cast<uint32_t>(src));
#pragma unroll
              for (int i = 0; i < 8; ++i) s[i] += ld_cluster_f32(a + i * kBM * 4);
            }
            const int64_t orig =
                has_plan ? (td.contig >= 0 ? td.contig + row : p.perm[td.row0 + row]) : td.row0 + row;
            uint4 o;
            o.x = pack_bf16x2(s[0], s[1]);
            o.y = pack_bf16x2(s[2], s[3]);
            o.z = pack_bf16x2(s[4], s[5]);
            o.w = pack_bf16x2(s[6], s[7]);
            *reinterpret_cast<uint4 *>(p.out + orig * p.N + col) = o;
          }
        }
      }
      cluster_barrier();  // no CTA leaves while another may still read its shared memory
    }
  }
}

}  // namespace lora
