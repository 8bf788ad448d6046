// The elementwise part of the feed-forward operators' backward passes.
//
//  k_act_dz<2> : gated; from dH and the saved G, U
//                  dG = bf16(dH U act'(G)),  dU = bf16(dH act(G))
//  k_act_dz<1> : one projection; from dY and the saved P, dP = bf16(dY act'(P)),
//                and the column sums of dP (dbias)
//                and, of the same tiles, the rank-r products dG Bg, dU Bu (dP B),
//                dZ = s times them: the gradients are written once and not read
//                back for dZ.
//  k_col_part  : the column sums of dY (dbias where there is no activation).
//
// All are HBM-bound (gated: 6 bytes read and 4 written per element of dH).
// Measured (MI355X): gated 4096 x 14336, rank 16, 112 to 115 us for 587 MB (5.2
// TB/s); one projection 2048 x 4096 with GELU, dbias and rank 32 23 us (50 MB: its
// 32 row slots are cut into 32 ranges of two steps, mostly prologue and epilogue).
// dG, dU and dP are rounded to bf16 because the large matrix products that
// follow take bf16 operands. The rank-r products take the rounding's remainder
// as a second bf16 operand too (two MFMAs for one, of which there are few), so
// that dZ, which is itself rounded to bf16 before dA and dX, carries one
// rounding and not two.
#pragma once

#include "act.hpp"
#include "norm.hpp"
#include "skinny.hpp"

namespace lora4 {
namespace actbwd {

constexpr int THREADS = 256;
constexpr float BF16_MAX = 0x1.FEp127f;

// ---------------------------------------------------------------------------
// Gradient of the activation, and dZ
// ---------------------------------------------------------------------------

struct DzParams {
  const uint16_t *dY;     // [M, N] (gated: dH)
  const uint16_t *pre;    // [M, P N]: G, U, or the pre-activation P
  const uint16_t *B;      // [groups P][N, r]
  int64_t M, N, Np;       // Np: N rounded up to 64
  int r, act;
  const int64_t *offsets;
  int groups;
  uint16_t *out;          // [M, P Np]: dG, dU, or dP; columns N .. Np - 1 are zero
  int steps;              // 64-column steps per range (blockIdx.y)
  float *part;            // [ranges][M][P r] fp32 partial sums of dG Bg, dU Bu (dP B)
  float *col_part;        // P = 1: [row slots][N] fp32 column sums of dP, or nullptr
  unsigned *zero;         // side job of block (0, 0): zero_n words set to 0
  int64_t zero_n;
};

// Workgroup: 64 rows x one range of 64-column steps. Per step each thread
// takes 2 pieces of 8 columns of each input (8 threads per 64-column row
// piece), writes the gradients out and, with their rounding remainders, into
// LDS, and the four waves (16 rows each) multiply them with the step's rows of
// B (LDS, read transposed). The next step's pieces are loaded before the
// products. TJ: 16-column blocks of the rank.
template <int P, int TJ>
__global__ __launch_bounds__(THREADS) void k_act_dz(DzParams p) {
  constexpr int BN = 16 * TJ, PPR = BN / 8;
  constexpr int NB = (64 * PPR + THREADS - 1) / THREADS;   // B pieces per thread and projection
  __shared__ __attribute__((aligned(16))) uint16_t As[P][2][64 * 64];   // value, remainder
  __shared__ __attribute__((aligned(16))) uint16_t Bs[P][64 * BN];
  __shared__ float cs[P == 1 ? 4 : 1][64];

  if (p.zero && blockIdx.x == 0 && blockIdx.y == 0)   // written through to memory
    for (int64_t i = threadIdx.x; i < p.zero_n; i += THREADS)
      __hip_atomic_store(&p.zero[i], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  const RowTile rt = map_row_tile_wave(blockIdx.x, 64, p.offsets, p.groups, p.M);
  if (rt.group < 0) return;
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int lr = lane & 15, lg = lane >> 4;
  const int all = (int)(p.Np >> 6);
  const int s0 = blockIdx.y * p.steps, s1 = min(s0 + p.steps, all);
  const uint16_t *B0 = p.B + (int64_t)rt.group * P * p.N * p.r;

  u32x4_t dy[2], pv[P][2], bv[P][NB];
  auto load = [&](int s) {
    const int64_t n0 = (int64_t)s * 64;
    const int cols = (int)min(p.N - n0, (int64_t)64);   // columns of this step below N
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = rt.row0 + 32 * h + (t >> 3);
      dy[h] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < P; ++j) pv[j][h] = u32x4_t{0u, 0u, 0u, 0u};
      if (row < rt.row_end && 8 * (t & 7) < cols) {
        dy[h] = norm::load_vec(p.dY + row * p.N + n0, t & 7, cols);
#pragma unroll
        for (int j = 0; j < P; ++j)
          pv[j][h] = norm::load_vec(p.pre + row * P * p.N + j * p.N + n0, t & 7, cols);
      }
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int idx = t + THREADS * i, n = idx / PPR, c = (idx % PPR) * 8;
        bv[j][i] = u32x4_t{0u, 0u, 0u, 0u};
        if (idx < 64 * PPR && n < cols && c < p.r)
          bv[j][i] = norm::load_vec(B0 + (j * p.N + n0 + n) * p.r, c >> 3, p.r);
      }
  };
  f32x4_t acc[P][TJ];
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int b = 0; b < TJ; ++b) acc[j][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (s0 < s1) load(s0);
  for (int s = s0; s < s1; ++s) {
    float sum[P == 1 ? 8 : 1] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rl = 32 * h + (t >> 3);
      u32x4_t d[P], hi[P], lo[P];   // the gradient; its two parts for dZ
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v0, d0, v1, d1;
        act_value_slope(norm::lo_f32(pv[0][h][e]), p.act, v0, d0);
        act_value_slope(norm::hi_f32(pv[0][h][e]), p.act, v1, d1);
        const float y0 = norm::lo_f32(dy[h][e]), y1 = norm::hi_f32(dy[h][e]);
        float a[P], b[P];
        if constexpr (P == 2) {
          a[0] = y0 * norm::lo_f32(pv[1][h][e]) * d0;
          b[0] = y1 * norm::hi_f32(pv[1][h][e]) * d1;
          a[1] = y0 * v0;
          b[1] = y1 * v1;
        } else {
          a[0] = y0 * d0;
          b[0] = y1 * d1;
          sum[2 * e] += a[0];   // (the column sums take the unrounded products)
          sum[2 * e + 1] += b[0];
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          d[j][e] = pack_bf16x2(a[j], b[j]);
          // dZ's first part is at most bf16's largest value, so that the second,
          // the rest, is finite where the gradient is (an infinite or NaN
          // gradient shows as an infinite or NaN rest)
          hi[j][e] = pack_bf16x2(__builtin_amdgcn_fmed3f(a[j], -BF16_MAX, BF16_MAX),
                                 __builtin_amdgcn_fmed3f(b[j], -BF16_MAX, BF16_MAX));
          lo[j][e] = pack_bf16x2(a[j] - norm::lo_f32(hi[j][e]), b[j] - norm::hi_f32(hi[j][e]));
        }
      }
      const int64_t row = rt.row0 + rl;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        lds_write_b128(As[j][0] + tile64_swz(rl, t & 7), hi[j]);
        lds_write_b128(As[j][1] + tile64_swz(rl, t & 7), lo[j]);
        if (row < rt.row_end)
          *reinterpret_cast<u32x4_t *>(p.out + row * P * p.Np + j * p.Np + (int64_t)s * 64 + 8 * (t & 7)) = d[j];
      }
    }
    if constexpr (P == 1) {
      if (p.col_part) {   // over the wave's 16 rows: lanes of equal t % 8
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum[e] += __shfl_xor(sum[e], 8);
          sum[e] += __shfl_xor(sum[e], 16);
          sum[e] += __shfl_xor(sum[e], 32);
        }
        if (lane < 8)
#pragma unroll
          for (int e = 0; e < 8; ++e) cs[wave][8 * lane + e] = sum[e];
      }
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int idx = t + THREADS * i, n = idx / PPR, c = idx % PPR;
        if (idx < 64 * PPR) lds_write_b128(Bs[j] + n * BN + ((c ^ skinny::bsw<BN>(n)) << 3), bv[j][i]);
      }
    __syncthreads();
    if (s + 1 < s1) load(s + 1);
    if constexpr (P == 1) {
      if (p.col_part && t < 64 && (int64_t)s * 64 + t < p.N)
        p.col_part[(int64_t)blockIdx.x * p.N + (int64_t)s * 64 + t] = (cs[0][t] + cs[1][t]) + (cs[2][t] + cs[3][t]);
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const u32x4_t a0 = lds_read_b128(As[j][0] + tile64_swz(16 * wave + lr, ks * 4 + lg));
        const u32x4_t a1 = lds_read_b128(As[j][1] + tile64_swz(16 * wave + lr, ks * 4 + lg));
        const int n = 32 * ks + 8 * lg + (lr >> 2);
#pragma unroll
        for (int b = 0; b < TJ; ++b) {
          const int c = 16 * b + (lr & 3) * 4;
          const u32x2_t lo = lds_read_tr16(Bs[j] + n * BN + (((c >> 3) ^ skinny::bsw<BN>(n)) << 3) + (c & 7));
          const u32x2_t hi =
              lds_read_tr16(Bs[j] + (n + 4) * BN + (((c >> 3) ^ skinny::bsw<BN>(n + 4)) << 3) + (c & 7));
          const u32x4_t w = {lo[0], lo[1], hi[0], hi[1]};
          acc[j][b] = mfma_16x16x32(a0, w, acc[j][b]);
          acc[j][b] = mfma_16x16x32(a1, w, acc[j][b]);
        }
      }
    __syncthreads();   // the tiles are rewritten by the next step
  }
  float *dst = p.part + (int64_t)blockIdx.y * p.M * P * p.r;
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int b = 0; b < TJ; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t row = rt.row0 + 16 * wave + 4 * lg + e;
        const int c = 16 * b + lr;
        if (row < rt.row_end && c < p.r) dst[row * P * p.r + j * p.r + c] = acc[j][b][e];
      }
}

// ---------------------------------------------------------------------------
// Column sums
// ---------------------------------------------------------------------------

struct ColParams {
  const uint16_t *dY;     // [M, N]
  int64_t M;
  int N;
  const int64_t *offsets;
  int groups;
  float *part;            // [groups][4 gridDim.y][N] partial column sums
};

constexpr int COL_BLOCK = 512;   // columns per block: 64 threads x 8

// Block: 512 columns x one of gridDim.y row ranges of group blockIdx.z; wave w
// takes rows w, w + 4, .. of the range.
static __global__ __launch_bounds__(THREADS) void k_col_part(ColParams p) {
  const int g = blockIdx.z;
  int64_t ga = 0, gb = p.M;
  if (p.offsets) {
    ga = p.offsets[g];
    gb = p.offsets[g + 1];
  }
  const int64_t per = (gb - ga + gridDim.y - 1) / gridDim.y;
  const int64_t m0 = ga + blockIdx.y * per, m1 = min(m0 + per, gb);
  const int wave = threadIdx.x >> 6, v = blockIdx.x * (COL_BLOCK / 8) + (threadIdx.x & 63);
  if (8 * v >= p.N) return;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
#pragma unroll 4
  for (int64_t row = m0 + wave; row < m1; row += 4) {
    const u32x4_t d = norm::load_vec(p.dY + row * p.N, v, p.N);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum[2 * e] += norm::lo_f32(d[e]);
      sum[2 * e + 1] += norm::hi_f32(d[e]);
    }
  }
  float *dst = p.part + (((int64_t)g * gridDim.y + blockIdx.y) * 4 + wave) * p.N;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (8 * v + e < p.N) dst[8 * v + e] = sum[e];
}

// dbias of one group from k_act_dz's column sums: the group's row slots of 64
// rows follow those of the groups before it. Block: 32 columns of group blockIdx.y.
static __global__ __launch_bounds__(1024) void k_col_sum_slots(const float *part, const int64_t *offsets, int groups,
                                                               int64_t M, int64_t N, uint16_t *out) {
  __shared__ float s[32][33];
  const int g = blockIdx.y, c = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;
  // slots of the groups before g, and of g
  int64_t first = 0, n = (M + 63) / 64;
  if (offsets) {
    for (int e = 0; e < g; ++e) first += (offsets[e + 1] - offsets[e] + 63) / 64;
    n = (offsets[g + 1] - offsets[g] + 63) / 64;
  }
  float a = 0.0f;
  if (col < N)
#pragma unroll 4
    for (int64_t i = q; i < n; i += 32) a += part[(first + i) * N + col];
  s[q][c] = a;
  __syncthreads();
  if (q == 0 && col < N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][c];
    out[g * N + col] = to_bf16(t);
  }
}

}  // namespace actbwd
}  // namespace lora4
