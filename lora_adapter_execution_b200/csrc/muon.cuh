// Orthogonalised updates of adapter factors (the Muon optimiser's step) over a
// rank-exact pool: adapter a's rows are a matrix U of r x d, r <= 256.
//
//   X0 = U / (|U|_F + eps);  X <- a·X + (b·A + c·A·A)·X,  A = X·X^T,  five times
//
// Every X is a polynomial of G0 = X0·X0^T times X0, so the d-long rows are read
// for one Gram matrix and for one product O = P·X0, and the five steps run on
// r x r matrices alone:
//
//   Q = a·I + b·G + c·G·G;   P <- P·Q;   G <- Q·G·Q      (all of them commute)
//
// Precision. A step multiplies a small singular value by a = 3.4445, so it grows
// a^2 = 11.86-fold in G per step, and so does any error G has there: 11.86^4 = 2e4-fold
// before the fifth step, and in the result the largest slope of P(g)·sqrt(g), 3.6e4 (at
// singular values of 0.004): an error of 2^-24 of |G| in G0 would be 2e-3 there. The Gram matrix and
// the r x r matrices are therefore held and multiplied in 64 bits (fp64 tensor
// MMAs); P is rounded once, to fp32, for the product with X0, whose own
// terms are fp32.
#pragma once

#include "common.cuh"
#include "fp8.cuh"   // ld_cluster_f32
#include "gemm.cuh"  // cluster_barrier, map_rank

namespace lora {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr double kNsAd = 3.4445, kNsBd = -4.7750, kNsCd = 2.0315;
constexpr double kNsEps = 1e-7;
constexpr int kNsSteps = 5;

// One adapter of a Muon context.
struct alignas(16) MuonAdapter {
  int32_t row0;     // first pool row
  int32_t rank;
  int32_t nt;       // 64-row tiles (ceil(rank / 64))
  int32_t index;    // the adapter's index (for `active`)
  int64_t gofs;     // its r x r matrices' offset in every matrix buffer, in doubles (pitch nt · 64)
  int64_t pofs;     // its partial Gram matrices' offset, in doubles
};
// One CTA's piece of a tiled pass over the adapters.
struct alignas(16) MuonItem {
  int32_t ad;     // index into the adapters
  int32_t ti, tj; // tile
  int32_t piece;
};

// The rows an update is made from: U = cg·g + cm·m (m null: U = g).
struct MuonInput {
  const float *g, *m;
  float cg, cm;
};
__device__ __forceinline__ float4 muon_u4(const MuonInput &in, int64_t ofs) {
  float4 g = *reinterpret_cast<const float4 *>(in.g + ofs);
  if (in.m) {
    const float4 m = *reinterpret_cast<const float4 *>(in.m + ofs);
    g.x = fmaf(in.cm, m.x, in.cg * g.x);
    g.y = fmaf(in.cm, m.y, in.cg * g.y);
    g.z = fmaf(in.cm, m.z, in.cg * g.z);
    g.w = fmaf(in.cm, m.w, in.cg * g.w);
  }
  return g;
}

// D (16 x 8) += A (16 x 4)·B (4 x 8) in fp64. Lane (g = lane / 4, t = lane % 4):
// a0, a1 = A[g][t], A[g + 8][t]; b = B[t][g]; d0, d1 = D[g][2t], D[g][2t + 1];
// d2, d3 the same in row g + 8.
__device__ __forceinline__ void dmma(double (&d)[4], double a0, double a1, double b) {
  asm volatile(
      "mma.sync.aligned.m16n8k4.row.col.f64.f64.f64.f64 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+d"(d[0]), "+d"(d[1]), "+d"(d[2]), "+d"(d[3])
      : "d"(a0), "d"(a1), "d"(b));
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void cp_async16_all(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// ------------------------------------------------------------------ momentum
// m' = beta·m + (1 - beta)·g over the rows of the listed adapters.
__global__ void __launch_bounds__(256)
    lora_muon_momentum_kernel(const MuonAdapter *__restrict__ ads, const int32_t *__restrict__ active, int64_t d,
                              const float *__restrict__ g, const float *m, float *m_out, float beta, float omb) {
  const MuonAdapter ad = ads[blockIdx.y];
  if (active && active[ad.index] == 0) return;
  const int64_t n4 = ad.rank * (d / 4);
  const int64_t base = ad.row0 * d;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n4; i += gridDim.x * 256ll) {
    const float4 gv = *reinterpret_cast<const float4 *>(g + base + 4 * i);
    float4 mv = *reinterpret_cast<const float4 *>(m + base + 4 * i);
    mv.x = fmaf(beta, mv.x, omb * gv.x);
    mv.y = fmaf(beta, mv.y, omb * gv.y);
    mv.z = fmaf(beta, mv.z, omb * gv.z);
    mv.w = fmaf(beta, mv.w, omb * gv.w);
    *reinterpret_cast<float4 *>(m_out + base + 4 * i) = mv;
  }
}

// ------------------------------------------------------------------ Gram tiles
// One 64 x 64 tile (ti <= tj) of U·U^T over one piece of the columns: 8 warps,
// each 16 x 32. Columns in chunks of 32, as doubles in shared memory (pitch 36:
// the eight rows and four columns of a fragment in different banks). Bound by the fp64
// tensor MMAs (64 multiply-adds a cycle and SM): 6 adapters of 256 x 4096 need 57 us of
// them; the whole orthogonalisation takes 334 us (301 in a graph; one chunk at a time: 419).
constexpr int kMuTile = 64;
constexpr int kMuChunk = 32;
// Columns of one piece of a Gram matrix: short ones spread a few adapters over the SMs,
// long ones leave fewer partial tiles (32 KB each) to store and add. Whole
// orthogonalisations in a graph, us, pieces of 256 / 384 / 512 / 640 / 1024: one
// 96 x 1024 73 / 81 / 87 / 95 / 117, one 256 x 4096 113 / 115 / 124 / 132 / 158, six of them
// 300 / 301 / 307 / 302 / 316, seven 349 / 355 / 360 / 363 / 356, six 256 x 11008 562 / 556 /
// 550 / 562 / 568, fifty 64 x 11008 391 / 382 / 382 / 378 / 404.
constexpr int kMuPieceCols = 384;
constexpr int kMuPitch = kMuChunk + 4;
__global__ void __launch_bounds__(256, 3)
    lora_muon_gram_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                          const int32_t *__restrict__ active, int64_t d, int64_t piece_cols, MuonInput in,
                          double *__restrict__ partial) {
  const MuonItem it = items[blockIdx.x];
  const MuonAdapter ad = ads[it.ad];
  pdl_launch_dependents();  // (launched the ordinary way: all before it is done)
  if (active && active[ad.index] == 0) return;
  __shared__ double sa[kMuTile][kMuPitch], sb[kMuTile][kMuPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int mi = (warp & 3) * 16, nj = (warp >> 2) * 32;
  const bool diag = it.ti == it.tj;
  double acc[4][4] = {};
  const int64_t c_end = min(d, (it.piece + 1) * piece_cols);
  // 64 rows x 32 columns per operand: 512 float4, two per thread; the next chunk's are
  // on their way while this one is multiplied
  float4 v[2], w[2];
  auto fetch = [&](int64_t c0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = threadIdx.x + 256 * u;
      const int row = e >> 3, c4 = (e & 7) * 4;
      const bool in_cols = c0 + c4 < c_end;
      v[u] = w[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in_cols && it.ti * kMuTile + row < ad.rank)
        v[u] = muon_u4(in, (ad.row0 + it.ti * kMuTile + row) * d + c0 + c4);
      if (!diag && in_cols && it.tj * kMuTile + row < ad.rank)
        w[u] = muon_u4(in, (ad.row0 + it.tj * kMuTile + row) * d + c0 + c4);
    }
  };
  fetch(it.piece * piece_cols);
  for (int64_t c0 = it.piece * piece_cols; c0 < c_end; c0 += kMuChunk) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = threadIdx.x + 256 * u;
      const int row = e >> 3, c4 = (e & 7) * 4;
      *reinterpret_cast<double2 *>(&sa[row][c4]) = make_double2(v[u].x, v[u].y);
      *reinterpret_cast<double2 *>(&sa[row][c4 + 2]) = make_double2(v[u].z, v[u].w);
      if (!diag) {
        *reinterpret_cast<double2 *>(&sb[row][c4]) = make_double2(w[u].x, w[u].y);
        *reinterpret_cast<double2 *>(&sb[row][c4 + 2]) = make_double2(w[u].z, w[u].w);
      }
    }
    __syncthreads();
    if (c0 + kMuChunk < c_end) fetch(c0 + kMuChunk);
    const double(*pb)[kMuPitch] = diag ? sa : sb;
#pragma unroll
    for (int k = 0; k < kMuChunk; k += 4) {
      const double a0 = sa[mi + g][k + t], a1 = sa[mi + g + 8][k + t];
#pragma unroll
      for (int j = 0; j < 4; ++j) dmma(acc[j], a0, a1, pb[nj + 8 * j + g][k + t]);
    }
    __syncthreads();
  }
  // partial tile [64][64] of this piece
  const int ntri = ad.nt * (ad.nt + 1) / 2;
  const int tri = it.ti * ad.nt - it.ti * (it.ti - 1) / 2 + (it.tj - it.ti);
  double *out = partial + ad.pofs + (static_cast<int64_t>(it.piece) * ntri + tri) * (kMuTile * kMuTile);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = nj + 8 * j + 2 * t;
    *reinterpret_cast<double2 *>(out + (mi + g) * kMuTile + col) = make_double2(acc[j][0], acc[j][1]);
    *reinterpret_cast<double2 *>(out + (mi + g + 8) * kMuTile + col) = make_double2(acc[j][2], acc[j][3]);
  }
}

// The launches from here to the application are short and each reads what the one
// before it wrote. They may be launched with programmatic serialization: they read their
// tables meanwhile and then wait, every CTA of them, so that the end of one launch means
// the end of all before it; the application, the last, lets nothing start early.

// kN values of a Gram tile, v[i] = the sum of its pieces at `at + i·step`, added in order,
// four pieces' loads in flight.
template <int kN>
__device__ __forceinline__ void muon_sum_pieces(double (&v)[kN], const double *at, int64_t step, int64_t stride,
                                                int pieces) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = 0.0;
  for (int p = 0; p < pieces; p += 4) {
    double x[4][kN];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < kN; ++i) x[q][i] = p + q < pieces ? at[(p + q) * stride + i * step] : 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] += x[q][i];
  }
}

// The pieces of an adapter's Gram tiles (a CTA an eighth of a tile) added in order and
// scaled to G0 = U·U^T / (|U|_F + eps)^2, both triangles, pitch nt·64 (zeros past the
// rank); |U|_F^2 is the trace. 1 / (|U|_F + eps) goes to inv[ad].
__global__ void __launch_bounds__(256)
    lora_muon_reduce_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                            const int32_t *__restrict__ active, int pieces, const double *__restrict__ partial,
                            double *__restrict__ G, double *__restrict__ inv) {
  const MuonItem it = items[blockIdx.x];
  const MuonAdapter ad = ads[it.ad];
  pdl_wait();
  pdl_launch_dependents();
  if (active && active[ad.index] == 0) return;
  const int ntri = ad.nt * (ad.nt + 1) / 2;
  constexpr int kT2 = kMuTile * kMuTile;
  __shared__ double red[256];
  const int64_t stride = static_cast<int64_t>(ntri) * kT2;  // from piece to piece
  // the trace, the same way in every CTA of the adapter (rank <= 256: a thread a term)
  double tr[1] = {0.0};
  if (static_cast<int>(threadIdx.x) < ad.rank) {
    const int i = threadIdx.x, ti = i / kMuTile, o = i % kMuTile;
    const int tri = ti * ad.nt - ti * (ti - 1) / 2;
    muon_sum_pieces(tr, partial + ad.pofs + static_cast<int64_t>(tri) * kT2 + o * kMuTile + o, 0, stride, pieces);
  }
  const int tri = it.ti * ad.nt - it.ti * (it.ti - 1) / 2 + (it.tj - it.ti);
  const int e0 = blockIdx.y * (kT2 / 8) + threadIdx.x;
  double v[2];
  muon_sum_pieces(v, partial + ad.pofs + static_cast<int64_t>(tri) * kT2 + e0, 256, stride, pieces);
  red[threadIdx.x] = tr[0];
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  const double s = 1.0 / (sqrt(red[0]) + kNsEps);
  if (it.ti == 0 && it.tj == 0 && blockIdx.y == 0 && threadIdx.x == 0) inv[it.ad] = s;
  const int pitch = ad.nt * kMuTile;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = e0 + 256 * u;
    const double x = v[u] * (s * s);
    const int i = it.ti * kMuTile + e / kMuTile, j = it.tj * kMuTile + e % kMuTile;
    G[ad.gofs + static_cast<int64_t>(i) * pitch + j] = x;
    if (it.ti != it.tj) G[ad.gofs + static_cast<int64_t>(j) * pitch + i] = x;
  }
}

// ------------------------------------------------------------------ r x r products
// One half, 32 x 16, of a 32 x 32 tile (ti <= tj in units of 32) of C = A·B for symmetric
// commuting matrices (so C is symmetric: the tile and its mirror are written); `poly`:
// C = a·I + b·A + c·A·B instead (A = B = G gives Q). Up to two products per launch
// (blockIdx.y). 4 warps, each 16 x 8 in four chains of MMAs (by k), added at the end; K in
// chunks of 32, three of them on their way by cp.async.
struct MuonProduct {
  const double *A, *B;
  double *C;
  int poly;
};
constexpr int kMuPt = 32;
constexpr int kMuPtStages = 4;
constexpr int kMuPtRows = kMuPt + kMuPt / 2;  // rows of A and B in a stage
constexpr int kMuPtSmem = kMuPtStages * kMuPtRows * kMuPitch * 8;
__global__ void __launch_bounds__(128)
    lora_muon_product_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                             const int32_t *__restrict__ active, MuonProduct p0, MuonProduct p1) {
  const MuonItem it = items[blockIdx.x >> 1];
  const MuonAdapter ad = ads[it.ad];
  pdl_wait();
  pdl_launch_dependents();
  if (active && active[ad.index] == 0) return;
  const MuonProduct p = blockIdx.y ? p1 : p0;
  extern __shared__ __align__(16) double mu_stages[];  // [stage][A's 32 rows, B's 16][kMuPitch]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int mi = (warp & 1) * 16, nj = (warp >> 1) * 8;
  const int half = (blockIdx.x & 1) * (kMuPt / 2);
  const int64_t pitch = ad.nt * kMuTile;
  const double *A = p.A + ad.gofs + it.ti * kMuPt * pitch;
  const double *B = p.B + ad.gofs + (it.tj * kMuPt + half) * pitch;  // rows of B for its columns: B is symmetric
  double acc[4][4] = {};
  const int kmax = (ad.rank + kMuPt - 1) / kMuPt * kMuPt;
  const int chunks = kmax / kMuPt;
  auto fetch = [&](int c) {  // one group a chunk, empty past the last
    if (c < chunks) {
      double *st = mu_stages + (c % kMuPtStages) * (kMuPtRows * kMuPitch);
#pragma unroll
      for (int u = 0; u < 6; ++u) {
        const int e = threadIdx.x + 128 * u;  // 512 pairs of A, 256 of B
        const int row = e >> 4, k = (e & 15) * 2;
        cp_async16_all(st + row * kMuPitch + k, (u < 4 ? A + row * pitch : B + (row - kMuPt) * pitch) + c * kMuPt + k);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int c = 0; c < kMuPtStages - 1; ++c) fetch(c);
  for (int c = 0; c < chunks; ++c) {
    cp_async_wait<kMuPtStages - 2>();
    __syncthreads();  // chunk c is here, and all are done with chunk c - 1, whose stage is filled next
    fetch(c + kMuPtStages - 1);
    const double(*sa)[kMuPitch] =
        reinterpret_cast<const double(*)[kMuPitch]>(mu_stages + (c % kMuPtStages) * (kMuPtRows * kMuPitch));
    const double(*sb)[kMuPitch] = sa + kMuPt;
#pragma unroll
    for (int k = 0; k < kMuPt; k += 4) {
      const double a0 = sa[mi + g][k + t], a1 = sa[mi + g + 8][k + t];
      dmma(acc[(k >> 2) & 3], a0, a1, sb[nj + g][k + t]);
    }
  }
  double *C = p.C + ad.gofs;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int row = it.ti * kMuPt + mi + g + (e >> 1) * 8;
    const int col = it.tj * kMuPt + half + nj + 2 * t + (e & 1);
    double v = (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]);
    if (p.poly)
      v = kNsCd * v + kNsBd * p.A[ad.gofs + row * pitch + col] + (row == col && row < ad.rank ? kNsAd : 0.0);
    C[row * pitch + col] = v;
    if (it.ti != it.tj) C[col * pitch + row] = v;
  }
}

// ------------------------------------------------------------------ application
// What becomes of O = P·X0: O itself, or w' = (1 - lr·wd)·w - lr·gain·O and its bf16 copy.
struct MuonOutput {
  float *O;             // orthogonalise: the result; null: the update
  const float *w;
  float *w_out;
  __nv_bfloat16 *pool;
  float keep;           // 1 - lr·wd
  float lr, rms;        // update w by -lr·gain·O, gain = rms·sqrt(max(rank, d)) (rms > 0) or 1
};
__device__ __forceinline__ void muon_store4(const MuonOutput &o, int64_t ofs, float step, float4 v, float4 w) {
  float4 n;
  n.x = fmaf(o.keep, w.x, -step * v.x);
  n.y = fmaf(o.keep, w.y, -step * v.y);
  n.z = fmaf(o.keep, w.z, -step * v.z);
  n.w = fmaf(o.keep, w.w, -step * v.w);
  *reinterpret_cast<float4 *>(o.w_out + ofs) = n;
  if (o.pool)
    *reinterpret_cast<uint2 *>(o.pool + ofs) = make_uint2(pack_bf16x2(n.x, n.y), pack_bf16x2(n.z, n.w));
}
__device__ __forceinline__ void muon_store4(const MuonOutput &o, int64_t ofs, float step, float4 v) {
  if (o.O) *reinterpret_cast<float4 *>(o.O + ofs) = v;
  else muon_store4(o, ofs, step, v, *reinterpret_cast<const float4 *>(o.w + ofs));
}
__device__ __forceinline__ float muon_step_size(const MuonOutput &o, int rank, int64_t d) {
  const float big = static_cast<float>(rank > d ? rank : d);
  return o.rms > 0.f ? o.lr * (o.rms * sqrtf(big)) : o.lr;
}

// 64 rows x 128 columns of O = P·X0: 256 threads, each 8 rows x 4 columns, ranks in
// chunks of 16, the next chunk on its way while this one is multiplied. Six 256 x 4096:
// 94 us, half the fp32 rate (8 x 8 per thread, two multiply-adds to an instruction and two
// buffers in shared memory, singly and together, took 94 to 97 us).
constexpr int kMuApCols = 128, kMuApK = 16;
__global__ void __launch_bounds__(256, 2)
    lora_muon_apply_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                           const int32_t *__restrict__ active, int64_t d, MuonInput in, const double *__restrict__ P,
                           const double *__restrict__ inv, MuonOutput out) {
  const MuonItem it = items[blockIdx.x];
  const MuonAdapter ad = ads[it.ad];
  pdl_wait();
  if (active && active[ad.index] == 0) return;
  __shared__ __align__(16) float sp[kMuApK][kMuTile];    // P^T: [k][row]
  __shared__ __align__(16) float su[kMuApK][kMuApCols];
  const int64_t pitch = ad.nt * kMuTile;
  const double s = inv[it.ad];
  const int64_t c0 = static_cast<int64_t>(it.piece) * kMuApCols;
  // a warp: 8 rows, its lanes the 32 groups of 4 columns
  const int tr = (threadIdx.x >> 5) * 8, tc = (threadIdx.x & 31) * 4;
  float4 acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  double pv[4];
  float4 uv[2];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = threadIdx.x + 256 * u;
      // P is symmetric: row k of P holds column k (zero past the rank within its tiles of 32)
      pv[u] = P[ad.gofs + (k0 + e / kMuTile) * pitch + it.ti * kMuTile + e % kMuTile];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = threadIdx.x + 256 * u;
      const int k = e >> 5, c = (e & 31) * 4;
      uv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < ad.rank && c0 + c < d) uv[u] = muon_u4(in, (ad.row0 + k0 + k) * d + c0 + c);
    }
  };
  fetch(0);
  for (int k0 = 0; k0 < ad.rank; k0 += kMuApK) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = threadIdx.x + 256 * u;
      sp[e / kMuTile][e % kMuTile] = static_cast<float>(pv[u] * s);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = threadIdx.x + 256 * u;
      *reinterpret_cast<float4 *>(&su[e >> 5][(e & 31) * 4]) = uv[u];
    }
    __syncthreads();
    if (k0 + kMuApK < ad.rank) fetch(k0 + kMuApK);
#pragma unroll
    for (int k = 0; k < kMuApK; ++k) {
      const float4 u = *reinterpret_cast<const float4 *>(&su[k][tc]);
      const float4 p0 = *reinterpret_cast<const float4 *>(&sp[k][tr]);
      const float4 p1 = *reinterpret_cast<const float4 *>(&sp[k][tr + 4]);
      const float av[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i].x = fmaf(av[i], u.x, acc[i].x);
        acc[i].y = fmaf(av[i], u.y, acc[i].y);
        acc[i].z = fmaf(av[i], u.z, acc[i].z);
        acc[i].w = fmaf(av[i], u.w, acc[i].w);
      }
    }
    __syncthreads();
  }
  const float step = muon_step_size(out, ad.rank, d);
  if (c0 + tc < d) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = it.ti * kMuTile + tr + i;
      if (row < ad.rank) muon_store4(out, (ad.row0 + row) * d + c0 + tc, step, acc[i]);
    }
  }
}

// ------------------------------------------------------------------ one launch per step
// Ranks up to 64 whose rows fit in shared memory: a cluster of CTAs per adapter,
// each CTA one slice of the columns, kept on chip from the first read to the
// result, so the rows cross HBM once (22 bytes an element for a step, 8 for an
// orthogonalisation). CTA: momentum and U of its slice (fp32, in shared memory),
// its slice's Gram matrix; the cluster's first CTA adds the slices' (through
// distributed shared memory, in order) and iterates; every CTA takes P from it and
// forms its slice of the result. One HBM pass, yet not bound by it: the phases of a
// cluster follow one another (read, Gram, iterate, apply) and the SM's other CTA fills
// the gaps only in part. 1000 adapters of ranks 1 to 21 at 4096 columns, a
// step: 320 us (154 us of bytes; the tiled passes: 2120 us; one launch per power-of-two
// rank: 495 us).
//
// Ranks are padded to a multiple of eight, R = 8·NB. The fp64 MMAs work on tiles of 16
// rows x 8 columns; of a symmetric matrix only those on or above the diagonal's 16 x 16
// blocks are formed and stored.
// Shared memory: U [8·NB][slice] fp32, column c of row i at c ^ ((i & 7) << 2) (a
// fragment's eight rows of four columns then lie in 32 different banks); three
// matrices of doubles, pitch RP = 8·NB rounded up to 16, column c of row i at
// c ^ ((i & 3) << 2) likewise. The space of the matrices first holds the warps'
// partial Gram matrices, as tiles in fragment order.
template <int NB>
struct MuF {
  static constexpr int M = (NB + 1) / 2;               // 16-row blocks
  static constexpr int RP = 16 * M;                    // pitch of the matrices
  static constexpr int R = 8 * NB;                     // padded rank
  static constexpr int kTiles = NB % 2 ? M * M : M * (M + 1);
  static constexpr int kPerP = (kTiles + 7) / 8;       // tiles per warp, one product
  static constexpr int kPerP2 = (2 * kTiles + 7) / 8;  // tiles per warp, two products
  static constexpr int kMat = RP * RP;                 // doubles
  static constexpr int kPart = kTiles * 128;           // doubles of a partial Gram matrix
  static constexpr int kBufs = NB <= 5 ? 8 : 4;        // partial Gram matrices at a time
  static constexpr int kMatBytes = (kBufs * kPart > 3 * kMat ? kBufs * kPart : 3 * kMat) * 8;
  static constexpr int kRows = NB <= 4 ? 8 : 16;       // rows per thread of the application
  static constexpr int kUn = NB == 1 ? 4 : 8;          // 16-byte loads in flight per thread and array
  static constexpr int kCtas = NB == 1 ? 4 : NB <= 4 ? 2 : 1;  // CTAs an SM should hold
  // The iteration: above rank 32 the cluster's CTAs share each product's tiles (rank
  // 64: 65,000 cycles in one CTA, bound by its fp64 MMAs); below it one CTA iterates
  // (a cluster barrier costs more than a product of rank 32).
  static constexpr bool kShared = NB >= 5;
  static constexpr int kCols4 = NB >= 5 ? 2 : 1;       // 4-column groups per thread of the application
};
// tile t of the list: row block i, column tile j (of 8), j = 2i .. NB - 1
template <int NB>
__device__ __forceinline__ void mu_tile(int t, int &i, int &j) {
  i = 0;
#pragma unroll
  for (int k = 0; k < MuF<NB>::M - 1; ++k)
    if (i == k && t >= NB - 2 * k) {
      t -= NB - 2 * k;
      i = k + 1;
    }
  j = 2 * i + t;
}
template <int NB>
__device__ __forceinline__ int mu_at(int row, int col) { return row * MuF<NB>::RP + (col ^ ((row & 3) << 2)); }

struct MuonFused {
  const float *g, *m;   // gradient and momentum in (m null: U = g)
  float *m_out;
  float beta, omb;
  int nesterov;
  int64_t d;
  int slice;            // columns per CTA, a multiple of 32
  int more;             // another launch of this step follows
};

// One tile of A·B for symmetric commuting operands, of which the 16 x 16 blocks on
// and above the diagonal are stored: a fragment of a block below it is read from its
// mirror (as free of bank conflicts: lanes (g, t) at column g ^ 4t of row t).
template <int NB>
__device__ __forceinline__ void mu_tile_product(const double *A, const double *B, int i, int j, int lane,
                                                double (&acc)[4]) {
  constexpr int RP = MuF<NB>::RP;
  const int g = lane >> 2, t = lane & 3;
  const int jb = j >> 1;
  const int sw = (g & 3) << 2, tw = t << 2;
  const double *a_row = A + (16 * i + g) * RP + t, *a_col = A + t * RP;
  const double *b_row = B + (8 * j + g) * RP + t, *b_col = B + t * RP;
  const int a_c0 = (16 * i + g) ^ tw, a_c1 = (16 * i + 8 + g) ^ tw, b_c = (8 * j + g) ^ tw;
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = 0.0;
#pragma unroll
  for (int k = 0; k < 8 * NB; k += 4) {
    const bool up_a = (k >> 4) >= i, up_b = (k >> 4) >= jb;
    const double a0 = *(up_a ? a_row + (k ^ sw) : a_col + k * RP + a_c0);
    const double a1 = *(up_a ? a_row + 8 * RP + (k ^ sw) : a_col + k * RP + a_c1);
    const double b = *(up_b ? b_row + (k ^ sw) : b_col + k * RP + b_c);
    dmma(acc, a0, a1, b);
  }
}
// ... and to shared memory; poly: c·acc + b·A + a·I instead
template <int NB>
__device__ __forceinline__ void mu_tile_write(double *C, const double *A, bool poly, int rank, int i, int j, int lane,
                                              const double (&acc)[4], uint32_t ncta) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 16 * i + g + 8 * h, col = 8 * j + 2 * t;
    const int o = mu_at<NB>(row, col);
    double2 v = make_double2(acc[2 * h], acc[2 * h + 1]);
    if (poly) {
      const double2 b = *reinterpret_cast<const double2 *>(A + o);
      v.x = kNsCd * v.x + kNsBd * b.x + (row == col && row < rank ? kNsAd : 0.0);
      v.y = kNsCd * v.y + kNsBd * b.y + (row == col + 1 && row < rank ? kNsAd : 0.0);
    }
    if constexpr (MuF<NB>::kShared) {
      const uint32_t a = smem_u32(C + o);
      for (uint32_t q = 0; q < ncta; ++q)
        asm volatile("st.shared::cluster.v2.f64 [%0], {%1, %2};" ::"r"(map_rank(a, q)), "d"(v.x), "d"(v.y) : "memory");
    } else {
      *reinterpret_cast<double2 *>(C + o) = v;
    }
  }
}
// The five steps: G (scaled) and the working matrices Q, P; P holds the result.
// A phase's tiles (of one product, or of two) are dealt to the 8 warps, or to those of
// all CTAs (kShared: each CTA holds all three matrices and writes its tiles to all).
template <int NB>
__device__ __forceinline__ void mu_iterate(double *G, double *Q, double *P, int rank, int warp, int lane,
                                           uint32_t cta, uint32_t ncta) {
  using F = MuF<NB>;
  const int first = F::kShared ? static_cast<int>(cta + ncta * warp) : warp;
  const int stride = F::kShared ? static_cast<int>(8 * ncta) : 8;
  auto sync = [&]() {
    if constexpr (F::kShared) cluster_barrier();
    else __syncthreads();
  };
#pragma unroll 1
  for (int step = 0; step < kNsSteps; ++step) {
    const bool last = step == kNsSteps - 1;
    {
      // Q = a·I + b·G + c·G·G (its last readers are behind a barrier); the first Q is P
      double a[F::kPerP][4];
#pragma unroll
      for (int q = 0; q < F::kPerP; ++q) {
        const int tile = first + stride * q;
        if (tile < F::kTiles) {
          int i, j;
          mu_tile<NB>(tile, i, j);
          mu_tile_product<NB>(G, G, i, j, lane, a[q]);
          mu_tile_write<NB>(Q, G, true, rank, i, j, lane, a[q], ncta);
          if (step == 0) mu_tile_write<NB>(P, G, true, rank, i, j, lane, a[q], ncta);
        }
      }
    }
    sync();
    {
      // T = Q·G in G's place, P·Q in P's: written once every read is done
      const int n_t = last ? 0 : F::kTiles, n = n_t + (step > 0 ? F::kTiles : 0);
      double a[F::kPerP2][4];
#pragma unroll
      for (int q = 0; q < F::kPerP2; ++q) {
        const int job = first + stride * q;
        if (job < n) {
          int i, j;
          mu_tile<NB>(job < n_t ? job : job - n_t, i, j);
          mu_tile_product<NB>(Q, job < n_t ? G : P, i, j, lane, a[q]);
        }
      }
      sync();
#pragma unroll
      for (int q = 0; q < F::kPerP2; ++q) {
        const int job = first + stride * q;
        if (job < n) {
          int i, j;
          mu_tile<NB>(job < n_t ? job : job - n_t, i, j);
          mu_tile_write<NB>(job < n_t ? G : P, nullptr, false, rank, i, j, lane, a[q], ncta);
        }
      }
      sync();
    }
    if (!last) {
      double a[F::kPerP][4];  // G = Q·T
#pragma unroll
      for (int q = 0; q < F::kPerP; ++q) {
        const int tile = first + stride * q;
        if (tile < F::kTiles) {
          int i, j;
          mu_tile<NB>(tile, i, j);
          mu_tile_product<NB>(Q, G, i, j, lane, a[q]);
        }
      }
      sync();
#pragma unroll
      for (int q = 0; q < F::kPerP; ++q) {
        const int tile = first + stride * q;
        if (tile < F::kTiles) {
          int i, j;
          mu_tile<NB>(tile, i, j);
          mu_tile_write<NB>(G, nullptr, false, rank, i, j, lane, a[q], ncta);
        }
      }
      sync();
    }
  }
}

template <int NB>
__global__ void __launch_bounds__(256, MuF<NB>::kCtas)
    lora_muon_fused_kernel(const MuonAdapter *__restrict__ ads, const int32_t *__restrict__ active, MuonFused p,
                           MuonOutput out) {
  using F = MuF<NB>;
  constexpr int RP = F::RP;
  extern __shared__ __align__(1024) uint8_t mu_smem[];
  double *mat = reinterpret_cast<double *>(mu_smem);
  float *us = reinterpret_cast<float *>(mu_smem + F::kMatBytes);
  uint32_t ncta, rank_in;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_in));
  // the launches of one step work on different adapters: the next one may start
  // once all of this one's CTAs run, and none ends before the one before it has
  if (p.more) pdl_launch_dependents();
  const MuonAdapter ad = ads[blockIdx.x / ncta];
  if (active && active[ad.index] == 0) {  // the whole cluster
    pdl_wait();
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = ad.rank;
  const int64_t c0 = static_cast<int64_t>(rank_in) * p.slice;
  const int nc4 = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(p.slice), p.d - c0)) / 4);
  const int64_t base = ad.row0 * p.d + c0;

  // ---- the slice's rows: momentum, U; where U is an input, straight to its place
  // (cp.async, all in flight at once)
  if (!p.m) {
    for (int e = threadIdx.x; e < r * nc4; e += 256) {
      const int row = e / nc4, c = 4 * (e - row * nc4);
      cp_async16_all(us + row * p.slice + (c ^ ((row & 7) << 2)), p.g + base + row * p.d + c);
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else {
    constexpr int kUn = F::kUn;
    const int total = r * nc4;
    int row = 0, c = static_cast<int>(threadIdx.x);
    if (nc4 > 0) {
      row = c / nc4;
      c -= row * nc4;
    }
    for (int e0 = threadIdx.x; e0 < total; e0 += 256 * kUn) {
      float4 gv[kUn], mv[kUn];
      int rr[kUn], cc[kUn];
#pragma unroll
      for (int u = 0; u < kUn; ++u) {
        rr[u] = row;
        cc[u] = c;
        if (e0 + 256 * u < total) {
          const int64_t o = base + row * p.d + 4 * c;
          gv[u] = *reinterpret_cast<const float4 *>(p.g + o);
          mv[u] = *reinterpret_cast<const float4 *>(p.m + o);
        }
        c += 256;
        while (c >= nc4) {
          c -= nc4;
          ++row;
        }
      }
#pragma unroll
      for (int u = 0; u < kUn; ++u) {
        if (e0 + 256 * u < total) {
          float4 v = gv[u];
          float4 m = mv[u];
          m.x = fmaf(p.beta, m.x, p.omb * v.x);
          m.y = fmaf(p.beta, m.y, p.omb * v.y);
          m.z = fmaf(p.beta, m.z, p.omb * v.z);
          m.w = fmaf(p.beta, m.w, p.omb * v.w);
          *reinterpret_cast<float4 *>(p.m_out + base + rr[u] * p.d + 4 * cc[u]) = m;
          if (p.nesterov) {
            v.x = fmaf(p.beta, m.x, p.omb * v.x);
            v.y = fmaf(p.beta, m.y, p.omb * v.y);
            v.z = fmaf(p.beta, m.z, p.omb * v.z);
            v.w = fmaf(p.beta, m.w, p.omb * v.w);
          } else {
            v = m;
          }
          *reinterpret_cast<float4 *>(us + rr[u] * p.slice + ((4 * cc[u]) ^ ((rr[u] & 7) << 2))) = v;
        }
      }
    }
  }
  __syncthreads();

  // ---- the slice's Gram matrix: each warp every eighth group of four columns, all
  // tiles (lane (g, t) needs the same values U[8 b + g][k + t] as A and as B fragments)
  {
    const int g = lane >> 2, t = lane & 3;
    double acc[F::kTiles][4] = {};
    for (int kk = warp; kk < nc4; kk += 8) {
      double v[2 * F::M];
#pragma unroll
      for (int b = 0; b < 2 * F::M; ++b)
        v[b] = b < NB && 8 * b + g < r ? static_cast<double>(us[(8 * b + g) * p.slice + ((4 * kk) ^ (g << 2)) + t]) : 0.0;
      int q = 0;
#pragma unroll
      for (int i = 0; i < F::M; ++i)
#pragma unroll
        for (int j = 2 * i; j < NB; ++j) dmma(acc[q++], v[2 * i], v[2 * i + 1], v[j]);
    }
    // the warps' sums, kBufs at a time: the upper half hands its sums to the lower one
    double2 *buf = reinterpret_cast<double2 *>(mat + (warp % F::kBufs) * F::kPart) + lane;
    if (F::kBufs == 4) {
      if (warp >= 4) {
#pragma unroll
        for (int q = 0; q < F::kTiles; ++q) {
          buf[(2 * q) * 32] = make_double2(acc[q][0], acc[q][1]);
          buf[(2 * q + 1) * 32] = make_double2(acc[q][2], acc[q][3]);
        }
      }
      __syncthreads();
      if (warp < 4) {
#pragma unroll
        for (int q = 0; q < F::kTiles; ++q) {
          const double2 x = buf[(2 * q) * 32], y = buf[(2 * q + 1) * 32];
          acc[q][0] += x.x, acc[q][1] += x.y, acc[q][2] += y.x, acc[q][3] += y.y;
        }
      }
    }
    if (warp < F::kBufs) {  // (over its own buffer, which it alone has read)
#pragma unroll
      for (int q = 0; q < F::kTiles; ++q) {
        buf[(2 * q) * 32] = make_double2(acc[q][0], acc[q][1]);
        buf[(2 * q + 1) * 32] = make_double2(acc[q][2], acc[q][3]);
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < F::kPart; e += 256) {
    double v = mat[e];
#pragma unroll
    for (int k = 1; k < F::kBufs; ++k) v += mat[k * F::kPart + e];
    mat[e] = v;
  }
  if (ncta > 1) cluster_barrier();
  else __syncthreads();
  float *pf = reinterpret_cast<float *>(mat);  // P as fp32 [RP][RP], in Q's place
  if (F::kShared || rank_in == 0) {
    // ---- G0, the iteration, P: every CTA (kShared) or the cluster's first
    static_assert(F::kPart <= 2 * F::kMat, "G's place is clear of the partial sums");
    double *Q = mat, *P = mat + F::kMat, *G = mat + 2 * F::kMat;
    for (int e = threadIdx.x; e < F::kPart; e += 256) {
      double w[8], v = 0.0;
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q) w[q] = q < ncta ? ld_cluster_f64(map_rank(smem_u32(mat + e), q)) : 0.0;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += w[q];
      // element (e & 1) of half h of lane ln of tile q
      const int ln = (e >> 1) & 31, h = (e >> 6) & 1;
      int i, j;
      mu_tile<NB>(e >> 7, i, j);
      G[mu_at<NB>(16 * i + 8 * h + (ln >> 2), 8 * j + 2 * (ln & 3) + (e & 1))] = v;
    }
    if (F::kShared) cluster_barrier();  // the partial sums are read: Q may take their place
    else __syncthreads();
    double tr = 0.0;
    for (int i = lane; i < r; i += 32) tr += G[mu_at<NB>(i, i)];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tr += __shfl_xor_sync(0xFFFFFFFFu, tr, o);
    const double inv = 1.0 / (sqrt(tr) + kNsEps);
    __syncthreads();
    for (int e = threadIdx.x; e < F::kMat; e += 256) G[e] *= inv * inv;  // (what is not part of a tile is never read)
    __syncthreads();
    mu_iterate<NB>(G, Q, P, r, warp, lane, rank_in, ncta);
    for (int e = threadIdx.x; e < F::kMat; e += 256) {
      const int row = e / RP, col = e % RP;
      const bool up = (col >> 4) >= (row >> 4);
      pf[e] = static_cast<float>(P[up ? mu_at<NB>(row, col) : mu_at<NB>(col, row)] * inv);
    }
  }
  if (!F::kShared && ncta > 1) {
    cluster_barrier();
    if (rank_in != 0) {
      const uint32_t src = map_rank(smem_u32(pf), 0);
      for (int e = threadIdx.x; e < F::kMat; e += 256) pf[e] = ld_cluster_f32(src + 4 * e);
    }
    // the first CTA stays until all have read P
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  __syncthreads();

  // ---- O = P·U of the slice: kRows rows x kCols4 groups of 4 columns per thread (P is
  // symmetric: row k holds column k)
  const float step = muon_step_size(out, r, p.d);
  const int ngrp = (r + F::kRows - 1) / F::kRows;
  const int nc = (nc4 + F::kCols4 - 1) / F::kCols4;
  for (int e = threadIdx.x; e < ngrp * nc; e += 256) {
    const int grp = e / nc;
    const int c = 4 * (e - grp * nc);
    float4 acc[F::kCols4][F::kRows];
#pragma unroll
    for (int h = 0; h < F::kCols4; ++h)
#pragma unroll
      for (int i = 0; i < F::kRows; ++i) acc[h][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    // (where registers allow, the weights are on their way while O is formed)
    constexpr bool kEarly = NB >= 2 && F::kRows == 8;
    float4 wv[kEarly ? 8 : 1];
    if (kEarly && !out.O) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (grp * 8 + i < r) wv[kEarly ? i : 0] = *reinterpret_cast<const float4 *>(out.w + base + (grp * 8 + i) * p.d + c);
    }
#pragma unroll 2
    for (int k = 0; k < r; ++k) {
      float4 u[F::kCols4];
#pragma unroll
      for (int h = 0; h < F::kCols4; ++h) {
        // (a second group past the slice's columns reads inside the row and is not stored)
        const int ch = min(c + 4 * h * nc, p.slice - 4);
        u[h] = *reinterpret_cast<const float4 *>(us + k * p.slice + (ch ^ ((k & 7) << 2)));
      }
      const float4 *pk = reinterpret_cast<const float4 *>(pf + k * RP + grp * F::kRows);
#pragma unroll
      for (int i4 = 0; i4 < F::kRows / 4; ++i4) {
        const float4 a = pk[i4];
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int h = 0; h < F::kCols4; ++h) {
            float4 &o = acc[h][4 * i4 + i];
            o.x = fmaf(av[i], u[h].x, o.x);
            o.y = fmaf(av[i], u[h].y, o.y);
            o.z = fmaf(av[i], u[h].z, o.z);
            o.w = fmaf(av[i], u[h].w, o.w);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < F::kCols4; ++h) {
      if (c + 4 * h * nc >= 4 * nc4) break;
#pragma unroll
      for (int i = 0; i < F::kRows; ++i) {
        const int row = grp * F::kRows + i;
        if (row < r) {
          const int64_t o = base + row * p.d + c + 4 * h * nc;
          if (kEarly && !out.O) muon_store4(out, o, step, acc[h][i], wv[kEarly ? i : 0]);
          else muon_store4(out, o, step, acc[h][i]);
        }
      }
    }
  }
  __syncwarp();
  if (!F::kShared && ncta > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  pdl_wait();
}

}  // namespace lora
