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
// a^2 = 12-fold in G per step, and so does any error G has there: an error of
// 2^-24 of |G| in G0 would be 5000 times as large by the fifth step. The Gram matrix and
// the r x r matrices are therefore held and multiplied in 64 bits (fp64 tensor
// MMAs); P is rounded once, to fp32, for the product with X0, whose own
// terms are fp32.
#pragma once

#include "common.cuh"

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
// the eight rows and four columns of a fragment in different banks).
constexpr int kMuTile = 64;
constexpr int kMuChunk = 32;
constexpr int kMuPieceCols = 512;  // columns of one piece of a Gram matrix
constexpr int kMuPitch = kMuChunk + 4;
__global__ void __launch_bounds__(256)
    lora_muon_gram_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                          const int32_t *__restrict__ active, int64_t d, int64_t piece_cols, MuonInput in,
                          double *__restrict__ partial) {
  const MuonItem it = items[blockIdx.x];
  const MuonAdapter ad = ads[it.ad];
  if (active && active[ad.index] == 0) return;
  __shared__ double sa[kMuTile][kMuPitch], sb[kMuTile][kMuPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int mi = (warp & 3) * 16, nj = (warp >> 2) * 32;
  const bool diag = it.ti == it.tj;
  double acc[4][4] = {};
  const int64_t c_end = min(d, (it.piece + 1) * piece_cols);
  for (int64_t c0 = it.piece * piece_cols; c0 < c_end; c0 += kMuChunk) {
    // 64 rows x 32 columns per operand: 512 float4, two per thread
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = threadIdx.x + 256 * u;
      const int row = e >> 3, c4 = (e & 7) * 4;
      const bool in_cols = c0 + c4 < c_end;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
      if (in_cols && it.ti * kMuTile + row < ad.rank)
        v = muon_u4(in, (ad.row0 + it.ti * kMuTile + row) * d + c0 + c4);
      sa[row][c4] = v.x, sa[row][c4 + 1] = v.y, sa[row][c4 + 2] = v.z, sa[row][c4 + 3] = v.w;
      if (!diag) {
        if (in_cols && it.tj * kMuTile + row < ad.rank)
          w = muon_u4(in, (ad.row0 + it.tj * kMuTile + row) * d + c0 + c4);
        sb[row][c4] = w.x, sb[row][c4 + 1] = w.y, sb[row][c4 + 2] = w.z, sb[row][c4 + 3] = w.w;
      }
    }
    __syncthreads();
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

// The pieces of an adapter's Gram tiles added in order and scaled to G0 =
// U·U^T / (|U|_F + eps)^2, both triangles, pitch nt·64 (zeros past the rank);
// |U|_F^2 is the trace. 1 / (|U|_F + eps) goes to inv[ad].
__global__ void __launch_bounds__(256)
    lora_muon_reduce_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                            const int32_t *__restrict__ active, int pieces, const double *__restrict__ partial,
                            double *__restrict__ G, double *__restrict__ inv) {
  const MuonItem it = items[blockIdx.x];
  const MuonAdapter ad = ads[it.ad];
  if (active && active[ad.index] == 0) return;
  const int ntri = ad.nt * (ad.nt + 1) / 2;
  constexpr int kT2 = kMuTile * kMuTile;
  __shared__ double red[256];
  // the trace, the same way in every CTA of the adapter
  double tr = 0.0;
  for (int i = threadIdx.x; i < ad.rank; i += 256) {
    const int ti = i / kMuTile, o = i % kMuTile;
    const int tri = ti * ad.nt - ti * (ti - 1) / 2;
    for (int p = 0; p < pieces; ++p)
      tr += partial[ad.pofs + (static_cast<int64_t>(p) * ntri + tri) * kT2 + o * kMuTile + o];
  }
  red[threadIdx.x] = tr;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  const double s = 1.0 / (sqrt(red[0]) + kNsEps);
  if (it.ti == 0 && it.tj == 0 && threadIdx.x == 0) inv[it.ad] = s;
  const int tri = it.ti * ad.nt - it.ti * (it.ti - 1) / 2 + (it.tj - it.ti);
  const int pitch = ad.nt * kMuTile;
  for (int e = threadIdx.x; e < kT2; e += 256) {
    double v = 0.0;
    for (int p = 0; p < pieces; ++p) v += partial[ad.pofs + (static_cast<int64_t>(p) * ntri + tri) * kT2 + e];
    v *= s * s;
    const int i = it.ti * kMuTile + e / kMuTile, j = it.tj * kMuTile + e % kMuTile;
    G[ad.gofs + static_cast<int64_t>(i) * pitch + j] = v;
    if (it.ti != it.tj) G[ad.gofs + static_cast<int64_t>(j) * pitch + i] = v;
  }
}

// ------------------------------------------------------------------ r x r products
// One 32 x 32 tile (ti <= tj in units of 32) of C = A·B for symmetric commuting
// matrices (so C is symmetric: the tile and its mirror are written); `poly`:
// C = a·I + b·A + c·A·B instead (A = B = G gives Q). Up to two products per launch
// (blockIdx.y). 4 warps, each 16 x 16; K in chunks of 32.
struct MuonProduct {
  const double *A, *B;
  double *C;
  int poly;
};
constexpr int kMuPt = 32;
__global__ void __launch_bounds__(128)
    lora_muon_product_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                             const int32_t *__restrict__ active, MuonProduct p0, MuonProduct p1) {
  const MuonItem it = items[blockIdx.x];
  const MuonAdapter ad = ads[it.ad];
  if (active && active[ad.index] == 0) return;
  const MuonProduct p = blockIdx.y ? p1 : p0;
  __shared__ double sa[kMuPt][kMuPitch], sb[kMuPt][kMuPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int mi = (warp & 1) * 16, nj = (warp >> 1) * 16;
  const int64_t pitch = ad.nt * kMuTile;
  const double *A = p.A + ad.gofs + it.ti * kMuPt * pitch;
  const double *B = p.B + ad.gofs + it.tj * kMuPt * pitch;  // rows of B for its columns: B is symmetric
  double acc[2][4] = {};
  const int kmax = (ad.rank + kMuPt - 1) / kMuPt * kMuPt;
  for (int k0 = 0; k0 < kmax; k0 += kMuPt) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = threadIdx.x + 128 * u;  // 512 double2 per operand
      const int row = e >> 4, c = (e & 15) * 2;
      *reinterpret_cast<double2 *>(&sa[row][c]) = *reinterpret_cast<const double2 *>(A + row * pitch + k0 + c);
      *reinterpret_cast<double2 *>(&sb[row][c]) = *reinterpret_cast<const double2 *>(B + row * pitch + k0 + c);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMuPt; k += 4) {
      const double a0 = sa[mi + g][k + t], a1 = sa[mi + g + 8][k + t];
      dmma(acc[0], a0, a1, sb[nj + g][k + t]);
      dmma(acc[1], a0, a1, sb[nj + 8 + g][k + t]);
    }
    __syncthreads();
  }
  double *C = p.C + ad.gofs;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = it.ti * kMuPt + mi + g + (e >> 1) * 8;
      const int col = it.tj * kMuPt + nj + 8 * j + 2 * t + (e & 1);
      double v = acc[j][e];
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
__device__ __forceinline__ void muon_store4(const MuonOutput &o, int64_t ofs, float step, float4 v) {
  if (o.O) {
    *reinterpret_cast<float4 *>(o.O + ofs) = v;
    return;
  }
  const float4 w = *reinterpret_cast<const float4 *>(o.w + ofs);
  float4 n;
  n.x = fmaf(o.keep, w.x, -step * v.x);
  n.y = fmaf(o.keep, w.y, -step * v.y);
  n.z = fmaf(o.keep, w.z, -step * v.z);
  n.w = fmaf(o.keep, w.w, -step * v.w);
  *reinterpret_cast<float4 *>(o.w_out + ofs) = n;
  if (o.pool)
    *reinterpret_cast<uint2 *>(o.pool + ofs) = make_uint2(pack_bf16x2(n.x, n.y), pack_bf16x2(n.z, n.w));
}
__device__ __forceinline__ float muon_step_size(const MuonOutput &o, int rank, int64_t d) {
  const float big = static_cast<float>(rank > d ? rank : d);
  return o.rms > 0.f ? o.lr * (o.rms * sqrtf(big)) : o.lr;
}

// 64 rows x 64 columns of O = P·X0: 256 threads, each 4 x 4, ranks in chunks of 32.
__global__ void __launch_bounds__(256)
    lora_muon_apply_kernel(const MuonAdapter *__restrict__ ads, const MuonItem *__restrict__ items,
                           const int32_t *__restrict__ active, int64_t d, MuonInput in, const double *__restrict__ P,
                           const double *__restrict__ inv, MuonOutput out) {
  const MuonItem it = items[blockIdx.x];
  const MuonAdapter ad = ads[it.ad];
  if (active && active[ad.index] == 0) return;
  __shared__ float sp[32][kMuTile + 4];  // P^T: [k][row]
  __shared__ __align__(16) float su[32][kMuTile];
  const int64_t pitch = ad.nt * kMuTile;
  const double s = inv[it.ad];
  const int tr = (threadIdx.x >> 4) * 4, tc = (threadIdx.x & 15) * 4;
  float acc[4][4] = {};
  const int64_t c0 = static_cast<int64_t>(it.piece) * kMuTile;
  for (int k0 = 0; k0 < ad.rank; k0 += 32) {
    for (int e = threadIdx.x; e < 32 * kMuTile; e += 256) {
      // P is symmetric: row k of P holds column k
      const int k = e / kMuTile, i = e % kMuTile;
      sp[k][i] = static_cast<float>(P[ad.gofs + (k0 + k) * pitch + it.ti * kMuTile + i] * s);
    }
    for (int e = threadIdx.x; e < 32 * kMuTile / 4; e += 256) {
      const int k = e / (kMuTile / 4), c = (e % (kMuTile / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < ad.rank && c0 + c < d) v = muon_u4(in, (ad.row0 + k0 + k) * d + c0 + c);
      *reinterpret_cast<float4 *>(&su[k][c]) = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float4 u = *reinterpret_cast<const float4 *>(&su[k][tc]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = sp[k][tr + i];
        acc[i][0] = fmaf(a, u.x, acc[i][0]);
        acc[i][1] = fmaf(a, u.y, acc[i][1]);
        acc[i][2] = fmaf(a, u.z, acc[i][2]);
        acc[i][3] = fmaf(a, u.w, acc[i][3]);
      }
    }
    __syncthreads();
  }
  const float step = muon_step_size(out, ad.rank, d);
  if (c0 + tc < d) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = it.ti * kMuTile + tr + i;
      if (row < ad.rank)
        muon_store4(out, (ad.row0 + row) * d + c0 + tc, step, make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]));
    }
  }
}

}  // namespace lora
