// The elementwise part of the feed-forward operators' backward passes.
//
//  k_gated_bwd : from dH and the saved G, U
//                  dG = bf16(dH U act'(G)),  dU = bf16(dH act(G))
//                and, of the same tiles, the rank-r products
//                  dG Bg, dU Bu   (dZ = s times them)
//                so dG and dU are written once and not read back for dZ.
//  k_act_bwd   : from dY and the saved P, dP = bf16(dY act'(P)), and the
//                column sums of dP (dbias).
//
// Both are HBM-bound (k_gated_bwd: 6 bytes read and 4 written per element of
// dH). dG, dU and dP are rounded to bf16 because the matrix products that
// follow take bf16 operands; dZ sees the same rounded values as dX and dB do.
#pragma once

#include "act.hpp"
#include "norm.hpp"
#include "skinny.hpp"

namespace lora4 {
namespace actbwd {

constexpr int THREADS = 256;

// ---------------------------------------------------------------------------
// Gated
// ---------------------------------------------------------------------------

struct GatedParams {
  const uint16_t *dH;     // [M, N]
  const uint16_t *GU;     // [M, 2 N]
  const uint16_t *B;      // [groups 2][N, r]
  int64_t M, N, Np;       // Np: N rounded up to 64
  int r, act;
  const int64_t *offsets;
  int groups;
  uint16_t *dGU;          // [M, 2 Np]; columns N .. Np - 1 of each half are zero
  int steps;              // 64-column steps per range (blockIdx.y)
  float *part;            // [ranges][M][2 r] fp32 partial sums of dG Bg, dU Bu
  unsigned *zero;         // side job of block (0, 0): zero_n words set to 0
  int64_t zero_n;
};

// Workgroup: 64 rows x one range of 64-column steps. Per step each thread
// takes 2 pieces of 8 columns of each of dH, G, U (8 threads per 64-column row
// piece), writes dG and dU out and into LDS, and the four waves (16 rows each)
// multiply them with the step's rows of Bg and Bu (LDS, read transposed). The
// next step's pieces are loaded before the products. TJ: 16-column blocks of
// the rank.
template <int TJ>
__global__ __launch_bounds__(THREADS) void k_gated_bwd(GatedParams p) {
  constexpr int BN = 16 * TJ, PPR = BN / 8;
  constexpr int NB = (64 * PPR + THREADS - 1) / THREADS;   // B pieces per thread and projection
  __shared__ __attribute__((aligned(16))) uint16_t As[2][64 * 64];
  __shared__ __attribute__((aligned(16))) uint16_t Bs[2][64 * BN];

  if (p.zero && blockIdx.x == 0 && blockIdx.y == 0)   // written through to memory
    for (int64_t i = threadIdx.x; i < p.zero_n; i += THREADS)
      __hip_atomic_store(&p.zero[i], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  const RowTile rt = map_row_tile(blockIdx.x, 64, p.offsets, p.groups, p.M);
  if (rt.group < 0) return;
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int lr = lane & 15, lg = lane >> 4;
  const int all = (int)(p.Np >> 6);
  const int s0 = blockIdx.y * p.steps, s1 = min(s0 + p.steps, all);
  const uint16_t *B0 = p.B + (int64_t)rt.group * 2 * p.N * p.r;

  u32x4_t dh[2], gt[2], up[2], bv[2][NB];
  auto load = [&](int s) {
    const int64_t n0 = (int64_t)s * 64;
    const int cols = (int)min(p.N - n0, (int64_t)64);   // columns of this step below N
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = rt.row0 + 32 * h + (t >> 3);
      dh[h] = u32x4_t{0u, 0u, 0u, 0u};
      gt[h] = dh[h];
      up[h] = dh[h];
      if (row < rt.row_end && 8 * (t & 7) < cols) {
        dh[h] = norm::load_vec(p.dH + row * p.N + n0, t & 7, cols);
        gt[h] = norm::load_vec(p.GU + row * 2 * p.N + n0, t & 7, cols);
        up[h] = norm::load_vec(p.GU + row * 2 * p.N + p.N + n0, t & 7, cols);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int idx = t + THREADS * i, n = idx / PPR, c = (idx % PPR) * 8;
        bv[j][i] = u32x4_t{0u, 0u, 0u, 0u};
        if (idx < 64 * PPR && n < cols && c < p.r)
          bv[j][i] = norm::load_vec(B0 + (j * p.N + n0 + n) * p.r, c >> 3, p.r);
      }
  };
  f32x4_t acc[2][TJ];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int b = 0; b < TJ; ++b) acc[j][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (s0 < s1) load(s0);
  for (int s = s0; s < s1; ++s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rl = 32 * h + (t >> 3);
      u32x4_t dg, du;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v0, d0, v1, d1;
        act_value_slope(norm::lo_f32(gt[h][e]), p.act, v0, d0);
        act_value_slope(norm::hi_f32(gt[h][e]), p.act, v1, d1);
        const float y0 = norm::lo_f32(dh[h][e]), y1 = norm::hi_f32(dh[h][e]);
        dg[e] = pack_bf16x2(y0 * norm::lo_f32(up[h][e]) * d0, y1 * norm::hi_f32(up[h][e]) * d1);
        du[e] = pack_bf16x2(y0 * v0, y1 * v1);
      }
      lds_write_b128(As[0] + tile64_swz(rl, t & 7), dg);
      lds_write_b128(As[1] + tile64_swz(rl, t & 7), du);
      const int64_t row = rt.row0 + rl;
      if (row < rt.row_end) {
        uint16_t *o = p.dGU + row * 2 * p.Np + (int64_t)s * 64 + 8 * (t & 7);
        *reinterpret_cast<u32x4_t *>(o) = dg;
        *reinterpret_cast<u32x4_t *>(o + p.Np) = du;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int idx = t + THREADS * i, n = idx / PPR, c = idx % PPR;
        if (idx < 64 * PPR) lds_write_b128(Bs[j] + n * BN + ((c ^ skinny::bsw<BN>(n)) << 3), bv[j][i]);
      }
    __syncthreads();
    if (s + 1 < s1) load(s + 1);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const u32x4_t a = lds_read_b128(As[j] + tile64_swz(16 * wave + lr, ks * 4 + lg));
        const int n = 32 * ks + 8 * lg + (lr >> 2);
#pragma unroll
        for (int b = 0; b < TJ; ++b) {
          const int c = 16 * b + (lr & 3) * 4;
          const u32x2_t lo = lds_read_tr16(Bs[j] + n * BN + (((c >> 3) ^ skinny::bsw<BN>(n)) << 3) + (c & 7));
          const u32x2_t hi =
              lds_read_tr16(Bs[j] + (n + 4) * BN + (((c >> 3) ^ skinny::bsw<BN>(n + 4)) << 3) + (c & 7));
          acc[j][b] = mfma_16x16x32(a, u32x4_t{lo[0], lo[1], hi[0], hi[1]}, acc[j][b]);
        }
      }
    __syncthreads();   // the tiles are rewritten by the next step
  }
  float *dst = p.part + (int64_t)blockIdx.y * p.M * 2 * p.r;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int b = 0; b < TJ; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t row = rt.row0 + 16 * wave + 4 * lg + e;
        const int c = 16 * b + lr;
        if (row < rt.row_end && c < p.r) dst[row * 2 * p.r + j * p.r + c] = acc[j][b][e];
      }
}

// ---------------------------------------------------------------------------
// Fused epilogue
// ---------------------------------------------------------------------------

struct ActParams {
  const uint16_t *dY;     // [M, N]
  const uint16_t *P;      // [M, N], or nullptr (no activation)
  int64_t M;
  int N, act;
  const int64_t *offsets;
  int groups;
  uint16_t *dP;           // [M, N], or nullptr (no activation: dP is dY)
  float *part;            // [groups][4 gridDim.y][N] partial column sums, or nullptr
};

constexpr int ACT_COLS = 512;   // columns per block: 64 threads x 8

// Block: 512 columns x one of gridDim.y row ranges of group blockIdx.z; wave w
// takes rows w, w + 4, .. of the range.
static __global__ __launch_bounds__(THREADS) void k_act_bwd(ActParams p) {
  const int g = blockIdx.z;
  int64_t ga = 0, gb = p.M;
  if (p.offsets) {
    ga = p.offsets[g];
    gb = p.offsets[g + 1];
  }
  const int64_t per = (gb - ga + gridDim.y - 1) / gridDim.y;
  const int64_t m0 = ga + blockIdx.y * per, m1 = min(m0 + per, gb);
  const int wave = threadIdx.x >> 6, v = blockIdx.x * (ACT_COLS / 8) + (threadIdx.x & 63);
  if (8 * v >= p.N) return;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
#pragma unroll 2
  for (int64_t row = m0 + wave; row < m1; row += 4) {
    u32x4_t d = norm::load_vec(p.dY + row * p.N, v, p.N);
    if (p.P) {
      const u32x4_t x = norm::load_vec(p.P + row * p.N, v, p.N);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v0, d0, v1, d1;
        act_value_slope(norm::lo_f32(x[e]), p.act, v0, d0);
        act_value_slope(norm::hi_f32(x[e]), p.act, v1, d1);
        const float a = norm::lo_f32(d[e]) * d0, b = norm::hi_f32(d[e]) * d1;
        sum[2 * e] += a;   // (the column sums take the unrounded products)
        sum[2 * e + 1] += b;
        d[e] = pack_bf16x2(a, b);
      }
      norm::store_vec(p.dP + row * p.N, v, p.N, d);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum[2 * e] += norm::lo_f32(d[e]);
        sum[2 * e + 1] += norm::hi_f32(d[e]);
      }
    }
  }
  if (p.part) {
    float *dst = p.part + (((int64_t)g * gridDim.y + blockIdx.y) * 4 + wave) * p.N;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * v + e < p.N) dst[8 * v + e] = sum[e];
  }
}

}  // namespace actbwd
}  // namespace lora4
